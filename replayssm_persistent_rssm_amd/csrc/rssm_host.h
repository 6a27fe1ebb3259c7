// rssm_host.h -- what the library's host-side files share: the error text of
// the calling thread, the verbose switch and small argument checks.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "rssm_materialize.h"

namespace rssm {

// Sets rssm_last_error()'s text and returns the status.
rssm_status fail(rssm_status st, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
void clear_error();
bool verbose();               // RSSM_MATERIALIZE_VERBOSE
const char* dtype_name(int d);

// Workgroups of 256 threads that one launch dimension takes (fewer than 2^32 threads).
constexpr int64_t kMaxWorkgroups = (int64_t(1) << 24) - 1;

template <typename T>
bool aligned(const T* p, size_t a) {
  return (reinterpret_cast<uintptr_t>(p) % a) == 0;
}

}  // namespace rssm
