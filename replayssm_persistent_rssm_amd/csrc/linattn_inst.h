// linattn_inst.h -- instance selection of the linear-attention kernels for one
// input dtype: state dtypes f32 / bf16 / f16, state widths 64 and 128.
#pragma once

#include "linattn_kernel.h"

namespace rssm {

enum : int { kLinChunk = 0, kLinFold = 1, kLinStep = 2 };

template <int IT, int ST, int N>
const void* linattn_fn(int which) {
  if (which == kLinChunk) return reinterpret_cast<const void*>(&linattn_chunk_kernel<IT, ST, N, false>);
  if (which == kLinFold) return reinterpret_cast<const void*>(&linattn_chunk_kernel<IT, ST, N, true>);
  return reinterpret_cast<const void*>(&linattn_step_kernel<IT, ST, N>);
}

template <int IT>
const void* linattn_pick(int which, int state_dtype, int dstate) {
  switch (state_dtype) {
    case kF32: return dstate == 64 ? linattn_fn<IT, kF32, 64>(which) : linattn_fn<IT, kF32, 128>(which);
    case kBF16: return dstate == 64 ? linattn_fn<IT, kBF16, 64>(which) : linattn_fn<IT, kBF16, 128>(which);
    case kF16: return dstate == 64 ? linattn_fn<IT, kF16, 64>(which) : linattn_fn<IT, kF16, 128>(which);
    default: return nullptr;
  }
}

}  // namespace rssm
