// pages_kernel.h -- gfx950 kernels of the page pool: extend, fork, release,
// compact and copy.
//
// The bookkeeping of a call is integers that depend on one another through prefix sums (an item's pages follow those of
// the items before it, a free page is found by its rank), so one workgroup of 1024 threads does it and leaves a plan in the
// workspace; the second kernel carries the plan out with the whole device.  Bytes move in tasks of 16 KiB that the
// workgroups take in turn: bound by memory where there is much to copy, by the two launches otherwise.
#pragma once

#include "mma_device.h"

namespace rssm {

struct PagesArgs {
  const int64_t* cache_ptrs;
  int32_t* table;
  int32_t* kv_len;
  int32_t* ref;
  const int32_t* src;
  const int32_t* dst;
  const int32_t* lengths;     // or null
  int32_t* status;
  int32_t* live;
  int32_t* claim;             // workspace: [num_rows] item that a row belongs to
  int32_t* first;             // [num_items] pages that the items before need
  int32_t* plan;              // [num_items] fork: its length, -1: nothing to do; extend: pages needed
  int32_t* fresh;             // [num_items] fork: the page of its own, -1: none
  int32_t* list;              // [num_pages] free pages; compact: holes, then the pages that move into them
  int32_t* moved;             // [num_pages] compact: new index of a page that moves
  int32_t* count;             // [2] compact: pages that move, pages in use
  int64_t table_stride, page_bytes, page_stride, token_bytes;
  int32_t num_items, num_rows, max_pages, num_pages, page_size, num_caches;
  int32_t chunks;             // tasks of kPagesChunk bytes a page
};

constexpr int kPlanBlock = 1024;
constexpr int kPlanPages = 16;          // page counts a thread looks at
constexpr int kPagesBlock = 256;
constexpr int kPagesChunk = 16384;      // bytes a task
constexpr int kPagesOk = 0, kPagesNone = 1, kPagesRefused = 2, kPagesShared = 3;

__device__ __forceinline__ int agent_load(const int32_t* p) {
  return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// Exclusive prefix sum over the workgroup, and the total.
struct PlanScan {
  int64_t wave[kPlanBlock / 64];
};
template <typename T>
__device__ __forceinline__ T plan_scan(PlanScan& lds, T v, T& total) {
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  T sum = v;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const T o = __shfl_up(sum, d);
    sum += lane >= d ? o : 0;
  }
  __syncthreads();                       // the previous use is over
  if (lane == 63) lds.wave[w] = sum;
  __syncthreads();
  T before = 0;
  total = 0;
#pragma unroll
  for (int i = 0; i < kPlanBlock / 64; ++i) {
    const T x = static_cast<T>(lds.wave[i]);
    before += i < w ? x : 0;
    total += x;
  }
  return before + sum - v;
}

typedef int i32x4u __attribute__((ext_vector_type(4), aligned(4)));

// Bits of the 16 page counts from `base` on that are 0 (free), and those inside the pool.
struct PlanMask { uint32_t free, in; };
__device__ __forceinline__ PlanMask plan_mask(const PagesArgs& a, int64_t base) {
  PlanMask m = {0, 0};
  if (base + kPlanPages <= a.num_pages) {
    m.in = (1u << kPlanPages) - 1;
#pragma unroll
    for (int i = 0; i < kPlanPages; i += 4) {
      const i32x4u v = *(const RSSM_GLOBAL i32x4u*)(a.ref + base + i);
      m.free |= (v[0] <= 0 ? 1u : 0u) << i | (v[1] <= 0 ? 2u : 0u) << i | (v[2] <= 0 ? 4u : 0u) << i | (v[3] <= 0 ? 8u : 0u) << i;
    }
  } else {
    for (int i = 0; i < kPlanPages && base + i < a.num_pages; ++i) {
      m.in |= 1u << i;
      m.free |= (gload(a.ref + base + i) <= 0 ? 1u : 0u) << i;
    }
  }
  return m;
}

__device__ __forceinline__ int pages_of(int64_t tokens, int page_size) {
  return static_cast<int>((tokens + page_size - 1) / page_size);
}

__device__ __forceinline__ int row_tokens(const PagesArgs& a, int row) {
  const int n = gload(a.kv_len + row);
  return n < 0 ? 0 : n;
}

// Extend and fork: who gets which pages.
template <bool FORK>
__global__ __launch_bounds__(kPlanBlock) void pages_plan_kernel(PagesArgs a) {
  __shared__ PlanScan lds;
  const int tid = threadIdx.x;
  // a row belongs to the first item that names it
  for (int i = tid; i < a.num_items; i += kPlanBlock) {
    const int r = gload(a.dst + i);
    if (r >= 0 && r < a.num_rows) __hip_atomic_store(a.claim + r, INT32_MAX, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  }
  __syncthreads();
  for (int i = tid; i < a.num_items; i += kPlanBlock) {
    const int r = gload(a.dst + i);
    if (r >= 0 && r < a.num_rows) atomicMin(a.claim + r, i);
  }
  __syncthreads();
  // what each item needs, and the pages that the items before it need
  int64_t wanted = 0;
  for (int base = 0; base < a.num_items; base += kPlanBlock) {
    const int i = base + tid;
    int need = 0;
    if (i < a.num_items) {
      const int r = gload(a.dst + i);
      int state = r >= 0 && r < a.num_rows && agent_load(a.claim + r) == i ? kPagesOk : kPagesRefused;
      int plan = -1;
      if (state == kPagesOk) {
        const int have = row_tokens(a, r);
        if constexpr (FORK) {
          const int s = gload(a.src + i);
          const int asked = a.lengths != nullptr ? gload(a.lengths + i) : INT32_MAX;
          if (s < 0 || s >= a.num_rows || asked < 0 || have != 0) {
            state = kPagesRefused;
          } else {
            const int64_t most = static_cast<int64_t>(a.max_pages) * a.page_size;
            const int n = row_tokens(a, s);
            plan = asked < n ? asked : n;
            plan = plan < most ? plan : static_cast<int>(most);
            need = plan % a.page_size != 0 ? 1 : 0;
          }
        } else {
          const int add = gload(a.lengths + i);
          const int64_t after = static_cast<int64_t>(have) + add;
          if (add < 0 || after > static_cast<int64_t>(a.max_pages) * a.page_size || after > INT32_MAX) {
            state = kPagesRefused;
          } else {
            const int held = pages_of(have, a.page_size);
            if (add > 0 && have % a.page_size != 0) {
              const int p = gload(a.table + r * a.table_stride + held - 1);
              if (p >= 0 && p < a.num_pages && gload(a.ref + p) > 1) state = kPagesShared;
            }
            if (state == kPagesOk) need = plan = pages_of(after, a.page_size) - held;
          }
        }
      }
      gstore(a.status + i, state);
      gstore(a.plan + i, plan);
    }
    int64_t total;                       // needs of a thousand rows may pass 32 bits
    const int64_t at = wanted + plan_scan<int64_t>(lds, need, total);
    if (i < a.num_items) gstore(a.first + i, static_cast<int32_t>(at < INT32_MAX ? at : INT32_MAX));
    wanted += total;
  }
  // free pages, lowest first, until there are enough
  int found = 0;
  for (int64_t base = 0; base < a.num_pages && found < wanted; base += kPlanBlock * kPlanPages) {
    const int64_t at = base + static_cast<int64_t>(tid) * kPlanPages;
    uint32_t free = at < a.num_pages ? plan_mask(a, at).free : 0u;
    int total;
    int k = found + plan_scan(lds, __builtin_popcount(free), total);
    for (; free != 0 && k < wanted; ++k, free &= free - 1)
      gstore(a.list + k, static_cast<int32_t>(at + __builtin_ctz(free)));
    found = static_cast<int>(found + total < wanted ? found + total : wanted);
  }
  __syncthreads();
  if constexpr (FORK) {
    for (int i = tid; i < a.num_items; i += kPlanBlock) {
      const int len = gload(a.plan + i);
      int page = -1;
      if (len >= 0) {
        const int r = gload(a.dst + i), at = gload(a.first + i);
        if (len % a.page_size != 0) {
          if (at < found) {
            page = gload(a.list + at);
            gstore(a.table + r * a.table_stride + len / a.page_size, page);
            gstore(a.ref + page, 1);
          } else {
            gstore(a.status + i, kPagesNone);
            gstore(a.plan + i, -1);
          }
        }
        if (len % a.page_size == 0 || page >= 0) gstore(a.kv_len + r, len);
      }
      gstore(a.fresh + i, page);
    }
  } else {
    // page k of the list goes to the last item whose pages start at or before k
    for (int k = tid; k < found; k += kPlanBlock) {
      int lo = 0, hi = a.num_items - 1;
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (gload(a.first + mid) <= k) lo = mid;
        else hi = mid - 1;
      }
      const int need = gload(a.plan + lo), at = gload(a.first + lo);
      if (need > 0 && at + static_cast<int64_t>(need) <= found) {
        const int r = gload(a.dst + lo), page = gload(a.list + k);
        gstore(a.table + r * a.table_stride + pages_of(row_tokens(a, r), a.page_size) + (k - at), page);
        gstore(a.ref + page, 1);
      }
    }
    __syncthreads();                     // rows keep their lengths until here
    for (int i = tid; i < a.num_items; i += kPlanBlock) {
      const int need = gload(a.plan + i);
      if (need < 0) continue;
      if (need > 0 && gload(a.first + i) + static_cast<int64_t>(need) > found) {
        gstore(a.status + i, kPagesNone);
      } else {
        const int r = gload(a.dst + i);
        gstore(a.kv_len + r, row_tokens(a, r) + gload(a.lengths + i));
      }
    }
  }
}

// One task: bytes [chunk kPagesChunk, ..) of a page, up to `bytes`.
__device__ __forceinline__ void copy_chunk(const PagesArgs& a, int cache, int from, int to, int chunk, int64_t bytes) {
  char* base = reinterpret_cast<char*>(sload(a.cache_ptrs + cache));
  const int64_t off = static_cast<int64_t>(chunk) * kPagesChunk;
  const char* s = base + from * a.page_stride + off;
  char* d = base + to * a.page_stride + off;
  const int n = static_cast<int>(bytes - off < kPagesChunk ? bytes - off : kPagesChunk);
  constexpr int kPer = kPagesChunk / (kPagesBlock * 16);
  u32x4 v[kPer];
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int at = (threadIdx.x + i * kPagesBlock) * 16;
    if (at < n) v[i] = ld<false, u32x4>(s + at);
  }
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int at = (threadIdx.x + i * kPagesBlock) * 16;
    if (at < n) st<false>(d + at, v[i]);
  }
}

__device__ __forceinline__ bool in_pool(const PagesArgs& a, int page) { return page >= 0 && page < a.num_pages; }

// Fork: the shared entries of each row, and the tokens of each page of its own.
__global__ __launch_bounds__(kPagesBlock) void pages_fork_kernel(PagesArgs a) {
  const int64_t per = 1 + static_cast<int64_t>(a.num_caches) * a.chunks, total = a.num_items * per;
  for (int64_t task = blockIdx.x; task < total; task += gridDim.x) {
    const int i = static_cast<int>(task / per), k = static_cast<int>(task - i * per);
    const int len = sload(a.plan + i);
    if (len < 0) continue;
    const int full = len / a.page_size, rest = len - full * a.page_size;
    const int32_t* from = a.table + sload(a.src + i) * a.table_stride;
    if (k == 0) {
      int32_t* to = a.table + sload(a.dst + i) * a.table_stride;
      for (int e = threadIdx.x; e < full; e += kPagesBlock) {
        const int page = gload(from + e);
        gstore(to + e, page);
        if (in_pool(a, page)) atomicAdd(a.ref + page, 1);
      }
    } else if (rest > 0) {
      const int cache = (k - 1) / a.chunks, chunk = (k - 1) - cache * a.chunks;
      const int64_t bytes = a.token_bytes > 0 ? rest * a.token_bytes : a.page_bytes;
      const int page = sload(from + full);
      if (chunk * static_cast<int64_t>(kPagesChunk) < bytes && in_pool(a, page)) copy_chunk(a, cache, page, sload(a.fresh + i), chunk, bytes);
    }
  }
}

// Release: a workgroup a row.  The minimum with the length that stays gives each page to one item alone, also when
// a row is named twice.
__global__ __launch_bounds__(kPagesBlock) void pages_release_kernel(PagesArgs a) {
  __shared__ int before;
  const int i = blockIdx.x;
  const int r = sload(a.dst + i), keep = a.lengths != nullptr ? sload(a.lengths + i) : 0;
  if (r < 0 || r >= a.num_rows || keep < 0) return;
  if (threadIdx.x == 0) before = atomicMin(a.kv_len + r, keep);
  __syncthreads();
  const int64_t most = a.max_pages;
  const int64_t held = pages_of(before < 0 ? 0 : before, a.page_size);
  int32_t* row = a.table + r * a.table_stride;
  for (int64_t e = pages_of(keep, a.page_size) + threadIdx.x; e < (held < most ? held : most); e += kPagesBlock) {
    const int page = gload(row + e);
    gstore(row + e, -1);
    if (in_pool(a, page)) atomicSub(a.ref + page, 1);
  }
}

// Compact: the pages that move, in order, and the counts after the moves.
__global__ __launch_bounds__(kPlanBlock) void pages_pack_kernel(PagesArgs a) {
  __shared__ PlanScan lds;
  const int tid = threadIdx.x;
  int used = 0;
  for (int64_t base = static_cast<int64_t>(tid) * kPlanPages; base < a.num_pages; base += kPlanBlock * kPlanPages) {
    const PlanMask m = plan_mask(a, base);
    used += __builtin_popcount(m.in & ~m.free);
  }
  int live;
  plan_scan(lds, used, live);
  // free pages before `live`, then pages in use from there on: as many of the one as of the other
  int listed = 0;
  for (int64_t base = 0; base < a.num_pages; base += kPlanBlock * kPlanPages) {
    const int64_t at = base + static_cast<int64_t>(tid) * kPlanPages;
    uint32_t pick = 0;
    if (at < a.num_pages) {
      const PlanMask m = plan_mask(a, at);
      const int64_t below = live - at;   // of these pages, so many lie before `live`
      const uint32_t low = below <= 0 ? 0u : below >= kPlanPages ? 0xffffffffu : (1u << below) - 1;
      pick = (m.free & low) | (m.in & ~m.free & ~low);
    }
    int total;
    int k = listed + plan_scan(lds, __builtin_popcount(pick), total);
    for (; pick != 0; ++k, pick &= pick - 1) gstore(a.list + k, static_cast<int32_t>(at + __builtin_ctz(pick)));
    listed += total;
  }
  __syncthreads();
  const int moves = listed / 2;
  for (int k = tid; k < moves; k += kPlanBlock) {
    const int hole = gload(a.list + k), page = gload(a.list + moves + k);
    gstore(a.moved + page, hole);
    gstore(a.ref + hole, gload(a.ref + page));
    gstore(a.ref + page, 0);
  }
  if (tid == 0) {
    gstore(a.count, moves);
    gstore(a.count + 1, live);
    gstore(a.live, live);
  }
}

// Compact: the rows' entries, then the bytes.
__global__ __launch_bounds__(kPagesBlock) void pages_move_kernel(PagesArgs a) {
  const int moves = sload(a.count), live = sload(a.count + 1);
  if (moves == 0) return;
  const int64_t per = static_cast<int64_t>(a.num_caches) * a.chunks, total = a.num_rows + moves * per;
  for (int64_t task = blockIdx.x; task < total; task += gridDim.x) {
    if (task < a.num_rows) {
      const int64_t held = pages_of(row_tokens(a, static_cast<int>(task)), a.page_size);
      int32_t* row = a.table + task * a.table_stride;
      for (int64_t e = threadIdx.x; e < (held < a.max_pages ? held : a.max_pages); e += kPagesBlock) {
        const int page = gload(row + e);
        if (page >= live && page < a.num_pages) gstore(row + e, gload(a.moved + page));
      }
    } else {
      const int64_t t = task - a.num_rows;
      const int m = static_cast<int>(t / per), k = static_cast<int>(t - m * per);
      const int cache = k / a.chunks;
      copy_chunk(a, cache, sload(a.list + moves + m), sload(a.list + m), k - cache * a.chunks, a.page_bytes);
    }
  }
}

__global__ __launch_bounds__(kPagesBlock) void pages_copy_kernel(PagesArgs a) {
  const int64_t per = static_cast<int64_t>(a.num_caches) * a.chunks, total = a.num_items * per;
  for (int64_t task = blockIdx.x; task < total; task += gridDim.x) {
    const int i = static_cast<int>(task / per), k = static_cast<int>(task - i * per), cache = k / a.chunks;
    const int from = sload(a.src + i), to = sload(a.dst + i);
    if (in_pool(a, from) && in_pool(a, to) && from != to) copy_chunk(a, cache, from, to, k - cache * a.chunks, a.page_bytes);
  }
}

}  // namespace rssm
