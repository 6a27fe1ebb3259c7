/*
 * rssm_block_norm.h -- C ABI of the norms around a block in
 * librssm_materialize (MI355X, gfx950): the gate and norm of a block's output,
 * its scaled addition to the residual stream and the norm before the next
 * block, in one pass.  For each row, with C channels in `groups` groups:
 *     u  = y * silu(z)                                      (no z: u = y)
 *     v  = u * post_weight / sqrt(mean of u^2 over its group + eps)   (no post_weight: v = u)
 *     r' = residual + residual_scale * channel_scale * v    (no channel_scale: 1)
 *     n  = r' * pre_weight / sqrt(mean of r'^2 over the row + eps)
 *
 * Plain C types only.  Every pointer is DEVICE memory owned by the caller;
 * the library allocates nothing and never synchronises.
 */
#ifndef RSSM_BLOCK_NORM_H
#define RSSM_BLOCK_NORM_H

#include <stdint.h>

#include "rssm_materialize.h" /* dtype codes, rssm_status, rssm_last_error */

#ifdef __cplusplus
extern "C" {
#endif

#define RSSM_BLOCK_NORM_MAX_CHANNELS 16384
#define RSSM_BLOCK_NORM_MAX_GROUPS 256

/*   rows              >= 0
 *   channels          C, a multiple of 8 in [8, RSSM_BLOCK_NORM_MAX_CHANNELS]
 *   groups            divides C into groups of a multiple of 8 channels, at most
 *                     RSSM_BLOCK_NORM_MAX_GROUPS (of the post norm only)
 *   input_dtype       y, z and normed: RSSM_F32 | RSSM_BF16 | RSSM_F16
 *   residual_dtype    residual and residual_out, likewise
 *   eps               >= 0
 *   *_row_stride      elements between rows; rows are dense inside */
typedef struct {
  int32_t rows;
  int32_t channels;
  int32_t groups;
  int32_t input_dtype;
  int32_t residual_dtype;
  float eps;
  float residual_scale;
  int64_t y_row_stride;
  int64_t z_row_stride;
  int64_t residual_row_stride;
  int64_t residual_out_row_stride;
  int64_t normed_row_stride;
} rssm_block_norm_desc;

/* z, post_weight, pre_weight and channel_scale ([channels] fp32) may be NULL; normed is
 * written from the fp32 r' before its rounding to the residual dtype, and may
 * be NULL (pre_weight then too).  residual_out may be residual itself, and
 * normed may be y itself.  Alignment: tensors 16 bytes, strides multiples of
 * 16 bytes, vectors 16 bytes. */
typedef struct {
  const void *y;
  const void *z;
  const void *residual;
  const float *post_weight;
  const float *pre_weight;
  const float *channel_scale;
  void *residual_out;
  void *normed;
} rssm_block_norm_tables;

/* Enqueue on `hip_stream`.  fp32 arithmetic; each output is rounded once. */
rssm_status rssm_block_norm(const rssm_block_norm_desc *desc, const rssm_block_norm_tables *tables, void *hip_stream);

#ifdef __cplusplus
}
#endif

#endif /* RSSM_BLOCK_NORM_H */
