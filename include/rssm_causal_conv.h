/*
 * rssm_causal_conv.h -- C ABI of the short causal convolution in front of a
 * state-space mixer in librssm_materialize (MI355X, gfx950): the form for
 * ragged prompts and the form for single tokens.  For one layer, channel c and
 * token t of a sequence, with W taps:
 *     y_t[c] = act(bias[c] + sum_{k < W} weight[k][c] x_{t-W+1+k}[c])
 * act is silu or nothing.  The inputs before the sequence's first row are the W - 1 rows
 * of its slot in the state pool, oldest first (zeros for a new sequence);
 * the call leaves the sequence's last W - 1 inputs there.
 *
 * Plain C types only.  Every pointer is DEVICE memory owned by the caller;
 * the library allocates nothing and never synchronises.
 */
#ifndef RSSM_CAUSAL_CONV_H
#define RSSM_CAUSAL_CONV_H

#include <stdint.h>

#include "rssm_materialize.h" /* dtype codes, rssm_status, rssm_last_error */

#ifdef __cplusplus
extern "C" {
#endif

/* Host-side scalars (both entry points).
 *   num_seqs           sequences (prompt form) or requests (single-token form) >= 0
 *   num_tokens         rows of x and y >= 0; the single-token form takes one row
 *                      per request and needs num_tokens == num_seqs
 *   channels           a multiple of 8 in [8, 2^20]
 *   width              W, taps in [2, 4]
 *   num_slots          slots of the state pool >= 1
 *   pad_slot_id        slot sentinel to skip (state and y rows left untouched)
 *   dtype              x, y and state: RSSM_F32 | RSSM_BF16 | RSSM_F16
 *   silu               1: act(v) = v / (1 + exp(-v)); 0: act(v) = v
 *   state_slot_stride  elements between slots, >= (W - 1) * channels
 *   *_token_stride     elements between rows; rows are dense inside, so that
 *                      views of one packed projection pass
 * One launch takes fewer than 2^24 workgroups: (num_tokens / 8 + num_seqs + 1) *
 * ceil(channels / 512) is below 2^26 (prompt form), num_seqs * ceil(channels / 512) likewise
 * (single-token form). */
typedef struct {
  int32_t num_seqs;
  int32_t num_tokens;
  int32_t channels;
  int32_t width;
  int32_t num_slots;
  int32_t pad_slot_id;
  int32_t dtype;
  int32_t silu;
  int64_t state_slot_stride;
  int64_t x_token_stride;
  int64_t y_token_stride;
} rssm_causal_conv_desc;

/* Device tensors:
 *   x, y        [num_tokens][channels] dtype
 *   weight      [W][channels] fp32
 *   bias        [channels] fp32 or NULL
 *   state       [slots][W - 1][channels] dtype, read and written
 *   slots       [num_seqs] int32
 *   seq_start   [num_seqs + 1] int32, ascending: sequence s owns rows
 *               seq_start[s] .. seq_start[s+1] - 1 (prompt form only)
 *   load_state  [num_seqs] int32 or NULL: 0 starts sequence s after zeros,
 *               otherwise (and with NULL) after its slot's rows (prompt form
 *               only).  An empty sequence stores its starting rows.
 * Device-metadata contract (not checked): live slots distinct; seq_start
 * ascending in [0, num_tokens].  As a guard against faults the kernels skip
 * slots outside [0, num_slots) and clamp seq_start to [0, num_tokens].  Rows of no sequence are left
 * untouched.  y may not alias x in the prompt form; in the single-token form it may be x itself.
 * Alignment: x, y, state, weight and bias 16 bytes, strides multiples of 16 bytes; the others 4 bytes. */
typedef struct {
  const void *x;
  const float *weight;
  const float *bias;
  void *y;
  void *state;
  const int32_t *slots;
  const int32_t *seq_start;
  const int32_t *load_state;
} rssm_causal_conv_tables;

/* Enqueue the prompt form on `hip_stream`.  fp32 arithmetic, one rounding of each output;
 * the state rows are the inputs' bytes. */
rssm_status rssm_causal_conv(const rssm_causal_conv_desc *desc, const rssm_causal_conv_tables *tables,
                             void *hip_stream);

/* Enqueue the single-token form on `hip_stream`: row b of x and y is request b's token. */
rssm_status rssm_causal_conv_step(const rssm_causal_conv_desc *desc, const rssm_causal_conv_tables *tables,
                                  void *hip_stream);

#ifdef __cplusplus
}
#endif

#endif /* RSSM_CAUSAL_CONV_H */
