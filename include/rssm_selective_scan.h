/*
 * rssm_selective_scan.h -- C ABI of the selective state-space scan in
 * librssm_materialize (MI355X, gfx950): a step size for each channel and a decay for each
 * channel and state (the first-generation mixer of hybrid decoders), for ragged prompts and for
 * single tokens.  For one layer, sequence s with state slot slots[s], channel c, state n and token t:
 *     d_t     = softplus(dt_t[c] + dt_bias[c])                (bias and softplus optional)
 *     h[c][n] <- exp(d_t A[c][n]) h[c][n] + d_t x_t[c] B_t[n]
 *     y_t[c]  =  sum_n h[c][n] C_t[n] + D[c] x_t[c], times silu(z_t[c])   (D and z optional)
 * with B and C of group c / (channels / groups).  The state after the last token goes back to the
 * slot, rounded once to the state dtype.
 *
 * Plain C types only.  Every pointer is DEVICE memory owned by the caller;
 * the library allocates nothing and never synchronises.
 */
#ifndef RSSM_SELECTIVE_SCAN_H
#define RSSM_SELECTIVE_SCAN_H

#include <stdint.h>

#include "rssm_materialize.h" /* dtype codes, rssm_status, rssm_last_error */

#ifdef __cplusplus
extern "C" {
#endif

/* Host-side scalars (both entry points).
 *   num_seqs           sequences (prompt form) or requests (single-token form) >= 0
 *   num_tokens         rows of x, dt, B, C, z and y >= 0; the single-token form
 *                      takes one row per request and needs num_tokens == num_seqs
 *   channels           a multiple of 8 in [8, 2^20]
 *   groups             divides channels, into multiples of 16 channels when above 1
 *   dstate             16, 32 or 64
 *   num_slots          slots of the state pool >= 1
 *   pad_slot_id        slot sentinel to skip (state and y rows left untouched)
 *   max_seq_len        longest sequence of the call, in [0, 2^30] (prompt form;
 *                      longer ones are cut to it)
 *   state_dtype        RSSM_F32 | RSSM_BF16 | RSSM_F16
 *   input_dtype        x, dt, B, C, z and y: RSSM_F32 | RSSM_BF16 | RSSM_F16
 *   dt_softplus        1: d = softplus(dt + bias); 0: d = dt + bias
 *   state_slot_stride  elements between slots, >= channels * dstate
 *   *_token_stride     elements between rows of each tensor (at most 2^24); rows are dense
 *                      inside, so that views of one packed projection pass
 *   workspace_bytes    bytes at tables->workspace
 * num_seqs * ceil(channels / 64) is below 2^24. */
typedef struct {
  int32_t num_seqs;
  int32_t num_tokens;
  int32_t channels;
  int32_t groups;
  int32_t dstate;
  int32_t num_slots;
  int32_t pad_slot_id;
  int32_t max_seq_len;
  int32_t state_dtype;
  int32_t input_dtype;
  int32_t dt_softplus;
  int32_t reserved; /* 0 */
  int64_t state_slot_stride;
  int64_t x_token_stride;
  int64_t dt_token_stride;
  int64_t B_token_stride;
  int64_t C_token_stride;
  int64_t z_token_stride;
  int64_t y_token_stride;
  int64_t workspace_bytes;
} rssm_selective_scan_desc;

/* Device tensors:
 *   state          [slots][channels][dstate] state dtype, read and written
 *   A              [channels][dstate] fp32 (-infinity: a state that keeps nothing of earlier tokens; steps below 2^-120
 *                  count as ones of size 0 or little more there, and a step of size 0 leaves every state as it is)
 *   D, dt_bias     [channels] fp32 each, or NULL
 *   x, dt, z, y    [num_tokens][channels] input dtype (z may be NULL)
 *   B, C           [num_tokens][groups][dstate] input dtype
 *   slots          [num_seqs] int32
 *   seq_start      [num_seqs + 1] int32, ascending: sequence s owns rows
 *                  seq_start[s] .. seq_start[s+1] - 1 (prompt form only)
 *   load_state     [num_seqs] int32 or NULL: 0 starts sequence s from a zero
 *                  state, otherwise (and with NULL) from its slot (prompt form
 *                  only).  An empty sequence stores its starting state.
 *   workspace      device memory of workspace_bytes, or NULL when 0 is needed
 * Device-metadata contract (not checked): live slots distinct; seq_start
 * ascending in [0, num_tokens].  As a guard against faults the kernels skip
 * slots outside [0, num_slots) and clamp seq_start to [0, num_tokens].
 * y may not alias an input.  Alignment: all floating tensors and the workspace 16
 * bytes, their strides multiples of 16 bytes; the others 4 bytes. */
typedef struct {
  void *state;
  const float *A;
  const float *D;
  const float *dt_bias;
  const void *x;
  const void *dt;
  const void *B;
  const void *C;
  const void *z;
  void *y;
  const int32_t *slots;
  const int32_t *seq_start;
  const int32_t *load_state;
  void *workspace;
} rssm_selective_scan_tables;

/* Workspace of the prompt form for these scalars, in bytes (0 when the sequences and channels fill the
 * device without splitting the token axis).  The single-token form needs none. */
rssm_status rssm_selective_scan_workspace(const rssm_selective_scan_desc *desc, int64_t *bytes);

/* Enqueue the prompt form on `hip_stream`.  fp32 arithmetic throughout, one rounding of each output.
 * Token t's output depends on tokens up to t only, non-finite inputs included.  With a split token axis
 * (workspace above 0) one launch reads the pool and the next one writes it, and the state that enters a
 * stretch is put together from the stretches before it; an infinity that a whole stretch decays to nothing
 * comes out as NaN there. */
rssm_status rssm_selective_scan(const rssm_selective_scan_desc *desc, const rssm_selective_scan_tables *tables,
                                void *hip_stream);

/* Enqueue the single-token form on `hip_stream`: row b of x, dt, B, C, z and y is request b's token.  fp32
 * arithmetic throughout; y is read from the fp32 state before its rounding. */
rssm_status rssm_selective_scan_step(const rssm_selective_scan_desc *desc, const rssm_selective_scan_tables *tables,
                                     void *hip_stream);

#ifdef __cplusplus
}
#endif

#endif /* RSSM_SELECTIVE_SCAN_H */
