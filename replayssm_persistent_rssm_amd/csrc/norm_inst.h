// norm_inst.h -- instance selection of the block-norm kernel for one input
// dtype: residual dtypes f32 / bf16 / f16, rows of up to 1, 2, 4 or 8 vectors a thread.
#pragma once

#include "norm_kernel.h"

namespace rssm {

template <int IT, int RT>
const void* norm_fn(int channels) {
  const int per = kNormBlock * 8;   // channels one vector a thread covers
  if (channels <= per) return reinterpret_cast<const void*>(&block_norm_kernel<IT, RT, 1>);
  if (channels <= 2 * per) return reinterpret_cast<const void*>(&block_norm_kernel<IT, RT, 2>);
  if (channels <= 4 * per) return reinterpret_cast<const void*>(&block_norm_kernel<IT, RT, 4>);
  return reinterpret_cast<const void*>(&block_norm_kernel<IT, RT, 8>);
}

template <int IT>
const void* norm_pick(int residual_dtype, int channels) {
  switch (residual_dtype) {
    case kF32: return norm_fn<IT, kF32>(channels);
    case kBF16: return norm_fn<IT, kBF16>(channels);
    case kF16: return norm_fn<IT, kF16>(channels);
    default: return nullptr;
  }
}

}  // namespace rssm
