/*
 * rssm_linear_attention.h -- C ABI of linear attention with a decay for each
 * head (the Mamba-2 recurrence) in librssm_materialize (MI355X, gfx950): the
 * chunked form for prompts and the recurrent form for single tokens.
 *
 * Both advance the state pools that the materialize operation and the decode
 * step read.  For one layer, sequence s with state slot slots[s] and tokens t:
 *     dt_t <- softplus(dt_raw_t[h] + dt_bias[h])      (bias and softplus optional; no dt: 1)
 *     S    <- exp(dt_t A_h) S + dt_t x_t B_t^T
 *     y_t  =  S C_t + D_h x_t, times silu(z_t)        (D and z optional)
 * with B and C of group g = h / heads_per_group.  The state after the last
 * token goes back to the slot, rounded once to the state dtype.
 *
 * Plain C types only.  Every pointer is DEVICE memory owned by the caller;
 * the library allocates nothing and never synchronises.
 */
#ifndef RSSM_LINEAR_ATTENTION_H
#define RSSM_LINEAR_ATTENTION_H

#include <stdint.h>

#include "rssm_materialize.h" /* dtype codes, rssm_status, rssm_last_error */

#ifdef __cplusplus
extern "C" {
#endif

/* Host-side scalars (both entry points).
 *   num_seqs           sequences (prompt form) or requests (single-token form) >= 0
 *   num_tokens         rows of x, B, C, dt, z and y >= 0; the single-token form
 *                      takes one row per request and needs num_tokens == num_seqs
 *   num_heads          H >= 1
 *   heads_per_group    divides H
 *   dim                64 or 128 (rows of a head's state)
 *   dstate             64 or 128 (columns)
 *   num_slots          slots of the state pool >= 1
 *   pad_slot_id        slot sentinel to skip (state and y rows left untouched)
 *   max_seq_len        longest sequence of the call, in [0, 2^30] (prompt form;
 *                      longer ones are cut to it)
 *   state_dtype        RSSM_F32 | RSSM_BF16 | RSSM_F16
 *   input_dtype        x, B, C, z and y: RSSM_F32 | RSSM_BF16 | RSSM_F16
 *   dt_softplus        1: dt = softplus(dt_raw + bias); 0: dt = dt_raw + bias
 *   state_slot_stride  elements between slots, >= H*dim*dstate
 *   *_token_stride     elements between rows of each tensor; rows are dense
 *                      inside, so that views of one packed projection pass
 *   workspace_bytes    bytes at tables->workspace
 * num_seqs * num_heads * dim / 64 is below 2^24. */
typedef struct {
  int32_t num_seqs;
  int32_t num_tokens;
  int32_t num_heads;
  int32_t heads_per_group;
  int32_t dim;
  int32_t dstate;
  int32_t num_slots;
  int32_t pad_slot_id;
  int32_t max_seq_len;
  int32_t state_dtype;
  int32_t input_dtype;
  int32_t dt_softplus;
  int64_t state_slot_stride;
  int64_t x_token_stride;
  int64_t B_token_stride;
  int64_t C_token_stride;
  int64_t dt_token_stride;
  int64_t z_token_stride;
  int64_t y_token_stride;
  int64_t workspace_bytes;
} rssm_linear_attention_desc;

/* Device tensors (G = H / heads_per_group):
 *   state          [slots][H][dim][dstate] state dtype, read and written
 *   A              [H] fp32 (-infinity: a head that keeps nothing; its dt must be above 0)
 *   D, dt_bias     [H] fp32 each, or NULL
 *   x, z, y        [num_tokens][H][dim] input dtype (z may be NULL)
 *   B, C           [num_tokens][G][dstate] input dtype
 *   dt             [num_tokens][H] fp32, or NULL (dt = 1; dt_bias must be NULL
 *                  and dt_softplus 0: a constant decay exp(A_h))
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
 * y may not alias an input.  Alignment: state, x, B, C, z, y and workspace 16
 * bytes, their strides multiples of 16 bytes; the others 4 bytes. */
typedef struct {
  void *state;
  const float *A;
  const float *D;
  const float *dt_bias;
  const void *x;
  const void *B;
  const void *C;
  const float *dt;
  const void *z;
  void *y;
  const int32_t *slots;
  const int32_t *seq_start;
  const int32_t *load_state;
  void *workspace;
} rssm_linear_attention_tables;

/* Workspace of the prompt form for these scalars, in bytes (0 when the
 * sequences and heads fill the device without splitting the token axis).
 * The single-token form needs none. */
rssm_status rssm_linear_attention_workspace(const rssm_linear_attention_desc *desc, int64_t *bytes);

/* Enqueue the prompt form on `hip_stream`.  Arithmetic: chunks of 64 tokens
 * on the matrix cores; the state and every sum are held in fp32.  The products
 * of the state update carry at least 22 bits for an fp32 state and 16 for a
 * 16-bit one; with fp16 inputs 22 for terms dt x down to 2^-29 of the largest
 * that the chunk adds to the same state row (decays counted), and 2^-51 of that
 * largest below.  16-bit inputs: for y, the decay-weighted scores and the chunk's
 * starting state are rounded once to the input dtype before their products.  fp16
 * scales the scores of a token, and each row of the state, by a power of two that
 * brings the largest to 2^12: nothing overflows, and entries below 2^-26 of that
 * largest are within 2^-37 of it.  Token t's output depends on tokens up to t
 * only, non-finite inputs included (in the state and the later tokens of its
 * heads an infinity may come out as NaN); a dt_raw of -infinity under softplus
 * skips its token. */
rssm_status rssm_linear_attention(const rssm_linear_attention_desc *desc, const rssm_linear_attention_tables *tables,
                                  void *hip_stream);

/* Enqueue the single-token form on `hip_stream`: row b of x, B, C, dt, z and y
 * is request b's token.  fp32 arithmetic throughout; y is read from the fp32
 * state before its rounding. */
rssm_status rssm_linear_attention_step(const rssm_linear_attention_desc *desc,
                                       const rssm_linear_attention_tables *tables, void *hip_stream);

#ifdef __cplusplus
}
#endif

#endif /* RSSM_LINEAR_ATTENTION_H */
