// pages_kernel.h -- gfx950 kernels of the page pool: extend, fork, release,
// compact and copy.
//
// The bookkeeping of a call is integers that depend on one another through prefix sums (an item's pages follow those of
// the items before it, a free page is found by its rank), so one workgroup of 1024 threads does it and leaves a plan in the
// workspace (3.3 us for 4 items, 5 to 6 for 128); the second kernel carries the plan out with the whole device.  Bytes move
// in tasks of 16 KiB that the workgroups take in turn: bound by memory where there is much to copy (128 forks in 32
// caches of 32 KiB pages, 67 MB in and out: 20 us), by the two launches otherwise.
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

// Sums that stop at 2^32 - 1: no pool has as many pages, so a sum that stopped asks for too many all the same.
__device__ __forceinline__ uint32_t add_sat(uint32_t a, uint32_t b) { return __builtin_elementwise_add_sat(a, b); }

// Inclusive prefix sum over the wavefront: within rows of 16 lanes, then the last lanes of rows 0 and 2 to rows 1 and 3, then
// lane 31 to the upper half.
__device__ __forceinline__ uint32_t wave_scan(uint32_t v) {
  v = add_sat(v, __builtin_amdgcn_update_dpp(0u, v, 0x111, 0xf, 0xf, true));
  v = add_sat(v, __builtin_amdgcn_update_dpp(0u, v, 0x112, 0xf, 0xf, true));
  v = add_sat(v, __builtin_amdgcn_update_dpp(0u, v, 0x114, 0xf, 0xf, true));
  v = add_sat(v, __builtin_amdgcn_update_dpp(0u, v, 0x118, 0xf, 0xf, true));
  v = add_sat(v, __builtin_amdgcn_update_dpp(0u, v, 0x142, 0xa, 0xf, false));
  return add_sat(v, __builtin_amdgcn_update_dpp(0u, v, 0x143, 0xc, 0xf, false));
}

// Exclusive prefix sum over a workgroup of B threads, and the total.  Successive calls alternate between two turns.
template <int B>
struct PlanScan {
  uint32_t wave[2][B / 64];
};
template <int B>
__device__ __forceinline__ uint32_t plan_scan(PlanScan<B>& lds, int turn, uint32_t v, uint32_t& total) {
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  const uint32_t sum = wave_scan(v);
  if (lane == 63) lds.wave[turn][w] = sum;
  __syncthreads();
  uint32_t before = 0;
  total = 0;
#pragma unroll
  for (int i = 0; i < B / 64; ++i) {
    const uint32_t x = lds.wave[turn][i];
    before = i < w ? add_sat(before, x) : before;
    total = add_sat(total, x);
  }
  const uint32_t prev = __builtin_amdgcn_update_dpp(0u, sum, 0x138, 0xf, 0xf, true);   // the lane before
  return add_sat(before, lane > 0 ? prev : 0u);
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

// Pages of 0 <= tokens < 2^31.
__device__ __forceinline__ int pages_of(int tokens, int page_size) {
  return static_cast<int>((static_cast<uint32_t>(tokens) + page_size - 1) / static_cast<uint32_t>(page_size));
}

__device__ __forceinline__ int row_tokens(const PagesArgs& a, int row) {
  const int n = gload(a.kv_len + row);
  return n < 0 ? 0 : n;
}

// What an item asks for: its status so far, its plan (fork: tokens, extend: pages; -1: nothing to do) and the
// pages it needs.  `mine`: it is the first item that names its row.
struct PlanAsk { int state, plan, need, have, held; };

template <bool FORK>
__device__ __forceinline__ PlanAsk plan_ask(const PagesArgs& a, bool mine, int row, int src, int length) {
  PlanAsk k = {kPagesRefused, -1, 0, 0, 0};
  if (!mine) return k;
  const int have = row_tokens(a, row);
  const int64_t most = static_cast<int64_t>(a.max_pages) * a.page_size;
  if constexpr (FORK) {
    if (src < 0 || src >= a.num_rows || length < 0) return k;
    int n = row_tokens(a, src);
    n = n < most ? n : static_cast<int>(most);
    if (have != 0) return k;
    k.state = kPagesOk;
    k.plan = length < n ? length : n;
    k.need = k.plan % a.page_size != 0 ? 1 : 0;
  } else {
    const int64_t after = static_cast<int64_t>(have) + length;
    if (length < 0 || after > most || after > INT32_MAX) return k;
    k.have = have;
    k.held = pages_of(have, a.page_size);
    if (length > 0 && have % a.page_size != 0) {
      const int p = gload(a.table + row * a.table_stride + k.held - 1);
      if (p >= 0 && p < a.num_pages && gload(a.ref + p) > 1) {
        k.state = kPagesShared;
        return k;
      }
    }
    k.state = kPagesOk;
    k.need = k.plan = pages_of(static_cast<int>(after), a.page_size) - k.held;
  }
  return k;
}

// Extend and fork of at most kPlanFew items, one a thread: everything but the tables' own entries stays in registers
// and LDS, and the first round of the search for free pages is requested before anything else.  B threads:
// 256 where one round of them sees the whole pool, 1024 otherwise.
constexpr int kPlanFew = 256;
constexpr int kPlanList = 2048;         // free pages kept in LDS, the rest in the workspace
constexpr int kPlanHash = 1024;

template <bool FORK, int B>
__global__ __launch_bounds__(B) void pages_plan_few_kernel(PagesArgs a) {
  __shared__ PlanScan<B> lds;
  __shared__ int rows[kPlanFew], hash[kPlanHash], held[kPlanFew], list[kPlanList];
  __shared__ uint32_t first[kPlanFew], needs[kPlanFew];
  const int tid = threadIdx.x, i = tid;
  const bool item = i < a.num_items;
  const int64_t at0 = static_cast<int64_t>(tid) * kPlanPages;
  uint32_t free = at0 < a.num_pages ? plan_mask(a, at0).free : 0u;
  int row = -1, src = 0, length = INT32_MAX;
  if (item) {
    row = gload(a.dst + i);
    if constexpr (FORK) src = gload(a.src + i);
    if (a.lengths != nullptr) length = gload(a.lengths + i);
  }
  for (int k = tid; k < kPlanHash; k += B) hash[k] = INT32_MAX;
  if (tid < kPlanFew) rows[tid] = row;
  __syncthreads();
  // a row belongs to the first item that names it: the lowest item of a slot decides unless another row shares the slot
  const bool known = item && row >= 0 && row < a.num_rows;
  if (known) atomicMin(&hash[row % kPlanHash], i);
  __syncthreads();
  bool mine = false;
  if (known) {
    const int k = hash[row % kPlanHash];
    mine = k == i;
    if (rows[k] != row) {
      mine = true;
      for (int m = 0; m < i; ++m) mine &= rows[m] != row;
    }
  }
  const PlanAsk ask = plan_ask<FORK>(a, mine, row, src, length);
  uint32_t wanted;
  const uint32_t at = plan_scan<B>(lds, 0, ask.need, wanted);
  if (tid < kPlanFew) {
    first[tid] = at;
    needs[tid] = ask.need;
    held[tid] = ask.held;
  }
  uint32_t found = 0;
  int turn = 1;
  for (int64_t base = 0; base < a.num_pages && found < wanted; base += B * kPlanPages, turn ^= 1) {
    const int64_t here = base + at0;
    if (base > 0) free = here < a.num_pages ? plan_mask(a, here).free : 0u;
    uint32_t total;
    uint32_t k = found + plan_scan<B>(lds, turn, __builtin_popcount(free), total);
    for (; free != 0 && k < wanted; ++k, free &= free - 1) {
      const int page = static_cast<int>(here + __builtin_ctz(free));
      if (k < kPlanList) list[k] = page;
      else gstore(a.list + k, page);
    }
    found = found + total < wanted ? found + total : wanted;
  }
  __syncthreads();
  const bool granted = ask.need == 0 || add_sat(at, ask.need) <= found;
  const int state = ask.state == kPagesOk && !granted ? kPagesNone : ask.state;
  if constexpr (FORK) {
    if (item) {
      int page = -1;
      if (state == kPagesOk) {
        if (ask.need > 0) {
          page = list[at];               // fewer items than kPlanList
          gstore(a.table + row * a.table_stride + ask.plan / a.page_size, page);
          gstore(a.ref + page, 1);
        }
        gstore(a.kv_len + row, ask.plan);
      }
      gstore(a.plan + i, state == kPagesOk ? ask.plan : -1);
      gstore(a.fresh + i, page);
      gstore(a.status + i, state);
    }
  } else {
    // page k of the list goes to the last item whose pages start at or before k
    for (uint32_t k = tid; k < found; k += B) {
      int lo = 0, hi = a.num_items - 1;
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (first[mid] <= k) lo = mid;
        else hi = mid - 1;
      }
      if (needs[lo] > 0 && add_sat(first[lo], needs[lo]) <= found) {
        const int page = k < kPlanList ? list[k] : gload(a.list + k);
        gstore(a.table + rows[lo] * a.table_stride + held[lo] + (k - first[lo]), page);
        gstore(a.ref + page, 1);
      }
    }
    if (item) {
      if (state == kPagesOk) gstore(a.kv_len + row, ask.have + length);
      gstore(a.status + i, state);
    }
  }
}

// Extend and fork of more items, in rounds.
template <bool FORK>
__global__ __launch_bounds__(kPlanBlock) void pages_plan_kernel(PagesArgs a) {
  __shared__ PlanScan<kPlanBlock> lds;
  int turn = 0;
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
    PlanAsk ask = {kPagesRefused, -1, 0, 0, 0};
    if (i < a.num_items) {
      const int r = gload(a.dst + i);
      const bool mine = r >= 0 && r < a.num_rows && agent_load(a.claim + r) == i;
      ask = plan_ask<FORK>(a, mine, r, FORK ? gload(a.src + i) : 0, a.lengths != nullptr ? gload(a.lengths + i) : INT32_MAX);
      gstore(a.status + i, ask.state);
      gstore(a.plan + i, ask.plan);
    }
    uint32_t total;
    const int64_t at = wanted + plan_scan<kPlanBlock>(lds, turn, ask.need, total);
    if (i < a.num_items) gstore(a.first + i, static_cast<int32_t>(at < INT32_MAX ? at : INT32_MAX));
    wanted += total;
    turn ^= 1;
  }
  // free pages, lowest first, until there are enough
  int found = 0;
  for (int64_t base = 0; base < a.num_pages && found < wanted; base += kPlanBlock * kPlanPages, turn ^= 1) {
    const int64_t at = base + static_cast<int64_t>(tid) * kPlanPages;
    uint32_t free = at < a.num_pages ? plan_mask(a, at).free : 0u;
    uint32_t total;
    int64_t k = found + static_cast<int64_t>(plan_scan<kPlanBlock>(lds, turn, __builtin_popcount(free), total));
    for (; free != 0 && k < wanted; ++k, free &= free - 1)
      gstore(a.list + k, static_cast<int32_t>(at + __builtin_ctz(free)));
    found = static_cast<int>(found + static_cast<int64_t>(total) < wanted ? found + static_cast<int64_t>(total) : wanted);
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

// One task: bytes [chunk kPagesChunk, ..) of a page, up to `bytes`.  NT: past the caches, for packing a pool (512 pages in
// 32 caches, 1.07 GB read and written: 200 us, 213 through them; branches, whose pages are used next, lose 7 % by it).
template <bool NT>
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
    if (at < n) v[i] = ld<NT, u32x4>(s + at);
  }
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int at = (threadIdx.x + i * kPagesBlock) * 16;
    if (at < n) st<NT>(d + at, v[i]);
  }
}

__device__ __forceinline__ bool in_pool(const PagesArgs& a, int page) { return page >= 0 && page < a.num_pages; }

// Fork: the shared entries of each row, and the tokens of each page of its own.
__global__ __launch_bounds__(kPagesBlock) void pages_fork_kernel(PagesArgs a) {
  const uint32_t chunks = a.chunks, per = 1 + a.num_caches * chunks, total = a.num_items * per;
  for (uint32_t task = blockIdx.x; task < total; task += gridDim.x) {
    const uint32_t i = task / per, k = task - i * per;
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
      const uint32_t cache = (k - 1) / chunks, chunk = (k - 1) - cache * chunks;
      const int64_t bytes = a.token_bytes > 0 ? rest * a.token_bytes : a.page_bytes;
      const int page = sload(from + full);
      if (chunk * static_cast<int64_t>(kPagesChunk) < bytes && in_pool(a, page)) copy_chunk<false>(a, cache, page, sload(a.fresh + i), chunk, bytes);
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
  const int held = pages_of(before < 0 ? 0 : before, a.page_size);
  int32_t* row = a.table + r * a.table_stride;
  for (int e = pages_of(keep, a.page_size) + threadIdx.x; e < (held < a.max_pages ? held : a.max_pages); e += kPagesBlock) {
    const int page = gload(row + e);
    gstore(row + e, -1);
    if (in_pool(a, page)) atomicSub(a.ref + page, 1);
  }
}

// Compact: the pages that move, in order, and the counts after the moves.
__global__ __launch_bounds__(kPlanBlock) void pages_pack_kernel(PagesArgs a) {
  __shared__ PlanScan<kPlanBlock> lds;
  const int tid = threadIdx.x;
  uint32_t used = 0;
  for (int64_t base = static_cast<int64_t>(tid) * kPlanPages; base < a.num_pages; base += kPlanBlock * kPlanPages) {
    const PlanMask m = plan_mask(a, base);
    used += __builtin_popcount(m.in & ~m.free);
  }
  uint32_t live;
  plan_scan<kPlanBlock>(lds, 0, used, live);
  // free pages before `live`, then pages in use from there on: as many of the one as of the other
  uint32_t listed = 0;
  int turn = 1;
  for (int64_t base = 0; base < a.num_pages; base += kPlanBlock * kPlanPages, turn ^= 1) {
    const int64_t at = base + static_cast<int64_t>(tid) * kPlanPages;
    uint32_t pick = 0;
    if (at < a.num_pages) {
      const PlanMask m = plan_mask(a, at);
      const int64_t below = static_cast<int64_t>(live) - at;   // of these pages, so many lie before `live`
      const uint32_t low = below <= 0 ? 0u : below >= kPlanPages ? 0xffffffffu : (1u << below) - 1;
      pick = (m.free & low) | (m.in & ~m.free & ~low);
    }
    uint32_t total;
    uint32_t k = listed + plan_scan<kPlanBlock>(lds, turn, __builtin_popcount(pick), total);
    for (; pick != 0; ++k, pick &= pick - 1) gstore(a.list + k, static_cast<int32_t>(at + __builtin_ctz(pick)));
    listed += total;
  }
  __syncthreads();
  const int moves = static_cast<int>(listed / 2);
  for (int k = tid; k < moves; k += kPlanBlock) {
    const int hole = gload(a.list + k), page = gload(a.list + moves + k);
    gstore(a.moved + page, hole);
    gstore(a.ref + hole, gload(a.ref + page));
    gstore(a.ref + page, 0);
  }
  if (tid == 0) {
    gstore(a.count, moves);
    gstore(a.count + 1, static_cast<int32_t>(live));
    gstore(a.live, static_cast<int32_t>(live));
  }
}

// Compact: the rows' entries, then the bytes.
__global__ __launch_bounds__(kPagesBlock) void pages_move_kernel(PagesArgs a) {
  const int moves = sload(a.count), live = sload(a.count + 1);
  if (moves == 0) return;
  const uint32_t rows = a.num_rows, chunks = a.chunks, per = a.num_caches * chunks, total = rows + moves * per;
  for (uint32_t task = blockIdx.x; task < total; task += gridDim.x) {
    if (task < rows) {
      const int held = pages_of(row_tokens(a, task), a.page_size);
      int32_t* row = a.table + task * a.table_stride;
      for (int e = threadIdx.x; e < (held < a.max_pages ? held : a.max_pages); e += kPagesBlock) {
        const int page = gload(row + e);
        if (page >= live && page < a.num_pages) gstore(row + e, gload(a.moved + page));
      }
    } else {
      const uint32_t t = task - rows, m = t / per, k = t - m * per, cache = k / chunks;
      copy_chunk<true>(a, cache, sload(a.list + moves + m), sload(a.list + m), k - cache * chunks, a.page_bytes);
    }
  }
}

__global__ __launch_bounds__(kPagesBlock) void pages_copy_kernel(PagesArgs a) {
  const uint32_t chunks = a.chunks, per = a.num_caches * chunks, total = a.num_items * per;
  for (uint32_t task = blockIdx.x; task < total; task += gridDim.x) {
    const uint32_t i = task / per, k = task - i * per, cache = k / chunks;
    const int from = sload(a.src + i), to = sload(a.dst + i);
    if (in_pool(a, from) && in_pool(a, to) && from != to) copy_chunk<false>(a, cache, from, to, k - cache * chunks, a.page_bytes);
  }
}

}  // namespace rssm
