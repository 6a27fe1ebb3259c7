// paged_inst.h -- instance selection of the paged-attention kernels for one
// dtype: head dims 64 and 128.
#pragma once

#include "paged_kernel.h"

namespace rssm {

enum : int { kPagedTile = 0, kPagedRow = 1, kPagedJoin = 2, kPagedJoinShare = 3 };

// Row blocks of 16 a wavefront of paged_tile_kernel holds: two share each K and V
// fragment read from LDS; fp32 operands take the registers of two 16-bit ones.
constexpr int paged_row_blocks(int dtype) { return dtype == kF32 ? 1 : 2; }

template <int IT, int D>
const void* paged_fn(int which) {
  if (which == kPagedTile) return reinterpret_cast<const void*>(&paged_tile_kernel<IT, D, paged_row_blocks(IT)>);
  if (which == kPagedRow) return reinterpret_cast<const void*>(&paged_row_kernel<IT, D>);
  if (which == kPagedJoin) return reinterpret_cast<const void*>(&paged_join_kernel<IT, D, false>);
  return reinterpret_cast<const void*>(&paged_join_kernel<IT, D, true>);
}

template <int IT>
const void* paged_pick(int which, int head_dim) {
  return head_dim == 64 ? paged_fn<IT, 64>(which) : paged_fn<IT, 128>(which);
}

}  // namespace rssm
