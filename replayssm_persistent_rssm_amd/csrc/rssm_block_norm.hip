// rssm_block_norm.hip -- host side of rssm_block_norm.h: argument checks and
// the launch on the caller's stream.
#include "rssm_block_norm.h"

#include <algorithm>
#include <cstdio>

#include "norm_inst.h"
#include "rssm_host.h"

namespace rssm {
const void* norm_f32_for(int residual_dtype, int channels);
const void* norm_bf16_for(int residual_dtype, int channels);
const void* norm_f16_for(int residual_dtype, int channels);
}  // namespace rssm

extern "C" rssm_status rssm_block_norm(const rssm_block_norm_desc* d, const rssm_block_norm_tables* t,
                                       void* hip_stream) {
  using namespace rssm;
  clear_error();
  if (d == nullptr) return fail(RSSM_ERR_INVALID_ARGUMENT, "desc is NULL");
  if (d->rows < 0) return fail(RSSM_ERR_INVALID_ARGUMENT, "rows must be >= 0 (got %d)", d->rows);
  if (d->channels < 8 || d->channels > RSSM_BLOCK_NORM_MAX_CHANNELS || d->channels % 8 != 0)
    return fail(RSSM_ERR_INVALID_ARGUMENT, "channels must be a multiple of 8 in [8, %d] (got %d)",
                RSSM_BLOCK_NORM_MAX_CHANNELS, d->channels);
  if (d->groups < 1 || d->groups > RSSM_BLOCK_NORM_MAX_GROUPS || d->channels % d->groups != 0 ||
      (d->channels / d->groups) % 8 != 0)
    return fail(RSSM_ERR_INVALID_ARGUMENT,
                "groups must be in [1, %d] and split channels into multiples of 8 (got %d groups of %d channels)",
                RSSM_BLOCK_NORM_MAX_GROUPS, d->groups, d->channels);
  for (int dt : {d->input_dtype, d->residual_dtype})
    if (dt < RSSM_F32 || dt > RSSM_F8E4M3) return fail(RSSM_ERR_INVALID_ARGUMENT, "unknown dtype %d", dt);
  if (d->input_dtype > RSSM_F16 || d->residual_dtype > RSSM_F16)
    return fail(RSSM_ERR_UNSUPPORTED, "input and residual dtypes must be f32, bf16 or f16 (got %s, %s)",
                dtype_name(d->input_dtype), dtype_name(d->residual_dtype));
  if (!(d->eps >= 0.0f)) return fail(RSSM_ERR_INVALID_ARGUMENT, "eps must be >= 0");
  const int64_t ie = d->input_dtype == RSSM_F32 ? 4 : 2, re = d->residual_dtype == RSSM_F32 ? 4 : 2;
  struct S { int64_t v, size; const char* n; };
  const S strides[] = {{d->y_row_stride, ie, "y_row_stride"}, {d->z_row_stride, ie, "z_row_stride"},
                       {d->residual_row_stride, re, "residual_row_stride"},
                       {d->residual_out_row_stride, re, "residual_out_row_stride"},
                       {d->normed_row_stride, ie, "normed_row_stride"}};
  for (const S& s : strides) {
    if (s.v < d->channels) return fail(RSSM_ERR_INVALID_ARGUMENT, "%s is below the dense row", s.n);
    if (s.v > (int64_t(1) << 31)) return fail(RSSM_ERR_INVALID_ARGUMENT, "%s exceeds 2^31 elements", s.n);
    if ((s.v * s.size) % 16 != 0) return fail(RSSM_ERR_INVALID_ARGUMENT, "%s must be a multiple of 16 bytes", s.n);
  }
  if (t == nullptr) return fail(RSSM_ERR_INVALID_ARGUMENT, "tables is NULL");
  if (d->rows == 0) return RSSM_OK;
  struct P { const void* p; const char* n; };
  const P need[] = {{t->y, "y"}, {t->residual, "residual"}, {t->residual_out, "residual_out"}};
  for (const P& e : need) {
    if (e.p == nullptr) return fail(RSSM_ERR_INVALID_ARGUMENT, "%s is NULL", e.n);
    if (!aligned(e.p, 16)) return fail(RSSM_ERR_INVALID_ARGUMENT, "%s is not 16-byte aligned", e.n);
  }
  const P opt[] = {{t->z, "z"}, {t->post_weight, "post_weight"}, {t->pre_weight, "pre_weight"},
                   {t->channel_scale, "channel_scale"}, {t->normed, "normed"}};
  for (const P& e : opt)
    if (e.p != nullptr && !aligned(e.p, 16)) return fail(RSSM_ERR_INVALID_ARGUMENT, "%s is not 16-byte aligned", e.n);
  if (t->normed == nullptr && t->pre_weight != nullptr)
    return fail(RSSM_ERR_INVALID_ARGUMENT, "pre_weight without normed");
  const void* fn = d->input_dtype == RSSM_F32    ? norm_f32_for(d->residual_dtype, d->channels)
                   : d->input_dtype == RSSM_BF16 ? norm_bf16_for(d->residual_dtype, d->channels)
                                                 : norm_f16_for(d->residual_dtype, d->channels);
  NormArgs a;
  a.y = static_cast<const char*>(t->y);
  a.z = static_cast<const char*>(t->z);
  a.residual = static_cast<const char*>(t->residual);
  a.post_weight = t->post_weight;
  a.pre_weight = t->pre_weight;
  a.channel_scale = t->channel_scale;
  a.residual_out = static_cast<char*>(t->residual_out);
  a.normed = static_cast<char*>(t->normed);
  a.y_stride = d->y_row_stride;
  a.z_stride = d->z_row_stride;
  a.r_stride = d->residual_row_stride;
  a.ro_stride = d->residual_out_row_stride;
  a.n_stride = d->normed_row_stride;
  a.C = d->channels;
  a.groups = d->groups;
  a.eps = d->eps;
  a.residual_scale = d->residual_scale;
  if (verbose())
    std::fprintf(stderr, "[rssm_block_norm] %s/%s rows=%d channels=%d groups=%d\n", dtype_name(d->input_dtype),
                 dtype_name(d->residual_dtype), d->rows, d->channels, d->groups);
  void* params[] = {&a};
  for (int64_t row = 0; row < d->rows; row += kMaxWorkgroups) {   // as many rows as one launch takes
    a.rows = static_cast<int32_t>(std::min<int64_t>(kMaxWorkgroups, d->rows - row));
    hipError_t e = hipLaunchKernel(fn, dim3(static_cast<unsigned>(a.rows)), dim3(kNormBlock), params, 0,
                                   static_cast<hipStream_t>(hip_stream));
    if (e != hipSuccess) return fail(RSSM_ERR_HIP, "launch of block_norm failed: %s", hipGetErrorString(e));
    a.y += a.rows * a.y_stride * ie;
    if (a.z != nullptr) a.z += a.rows * a.z_stride * ie;
    a.residual += a.rows * a.r_stride * re;
    a.residual_out += a.rows * a.ro_stride * re;
    if (a.normed != nullptr) a.normed += a.rows * a.n_stride * ie;
  }
  return RSSM_OK;
}
