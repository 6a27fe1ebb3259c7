// scan_inst.h -- instance selection of the selective-scan kernels for one input dtype.
#pragma once

#include "scan_kernel.h"

namespace rssm {

enum : int { kScanMain = 0, kScanFold = 1, kScanStepOne = 2, kScanStepTwo = 3, kScanShort = 4 };

template <int IT, int N>
const void* scan_fn(int which, int state_dtype) {
  if (which == kScanMain) return reinterpret_cast<const void*>(&scan_kernel<IT, N, false>);
  if (which == kScanFold) return reinterpret_cast<const void*>(&scan_kernel<IT, N, true>);
  if (which == kScanShort) return reinterpret_cast<const void*>(&scan_short_kernel<IT, N>);
  const bool two = which == kScanStepTwo;
  switch (state_dtype) {
    case kF32:
      return two ? reinterpret_cast<const void*>(&scan_step_kernel<IT, kF32, N, 2>)
                  : reinterpret_cast<const void*>(&scan_step_kernel<IT, kF32, N, 1>);
    case kBF16:
      return two ? reinterpret_cast<const void*>(&scan_step_kernel<IT, kBF16, N, 2>)
                  : reinterpret_cast<const void*>(&scan_step_kernel<IT, kBF16, N, 1>);
    default:
      return two ? reinterpret_cast<const void*>(&scan_step_kernel<IT, kF16, N, 2>)
                  : reinterpret_cast<const void*>(&scan_step_kernel<IT, kF16, N, 1>);
  }
}

template <int IT>
const void* scan_pick(int which, int state_dtype, int dstate) {
  return dstate == 16 ? scan_fn<IT, 16>(which, state_dtype)
         : dstate == 32 ? scan_fn<IT, 32>(which, state_dtype) : scan_fn<IT, 64>(which, state_dtype);
}

}  // namespace rssm
