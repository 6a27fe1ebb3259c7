// paged_kernel.h -- gfx950 kernels of the append to a paged key/value cache
// and of causal attention over it.
//
// Rows of a tile are (new token, query head of the group) pairs of one
// key/value head: row R is token R / group, head R % group.  Per tile of keys,
// transposed like the linear-attention kernel (mma_device.h):
//   S^T[j][i] = K_j . Q_i        A = K rows, Bm = Q rows (registers)
//   P = exp2(c S - m)            column i is the lane's: maximum and sum need two
//                                exchanges between the four lane groups
//   O^T[d][i] += V^T P           A = V columns (transposing LDS read), Bm = P
// with the running maximum m and sum l of each row (one pass over K and V).
//  * paged_tile_kernel: many rows.  4 wavefronts x 16 RB rows share the K and
//    V tiles of 64 tokens, double-buffered in LDS; the next tile is loaded
//    into registers while the current one is computed.
//  * paged_row_kernel: at most 16 rows (single-token decoding).  Bound by
//    reading the cache, so every wavefront streams its own tiles of 32
//    tokens, K straight into operand registers and V through its own part of LDS,
//    without barriers; the four partial results are joined in LDS.
// When there are few row tiles, the tiles of keys are split over workgroups and
// paged_join_kernel joins the partial outputs in a fixed order.
//
// paged_tile_kernel is bound by issue and LDS: 2,048 new bf16 tokens over 16,384, 32 query and 8
// key/value heads of 128: 0.597 ms with the append, 862 TFLOP/s, the vector ALUs busy 42% of the time, LDS
// 59%, the matrix cores 37%.  Leaving out the staging of K and V took
// a third off while the page table was still searched by every wavefront, which is why one wavefront a tile
// does it now (0.685 -> 0.594 ms); leaving out the exponentials took 5%, the second product 18%.  Eight
// wavefronts a tile, with or without half of them half a tile behind, ran 6% slower than
// four; four row blocks a wavefront (one wavefront a SIMD) 55% slower.
// paged_row_kernel is bound by memory: 64 requests, 1 to 8,192 tokens, 32 / 8 heads of 128, pages of
// 16: 0.212 ms with the append, 5.2 TB/s of cache read.
#pragma once

#include "mma_device.h"

namespace rssm {

struct PagedArgs {
  char* k;
  char* v;
  const char* k_new;
  const char* v_new;
  const char* q;
  char* out;
  float* lse;                 // or null
  const int32_t* table;
  const int32_t* seq_start;
  const int32_t* kv_len;
  float* part_o;              // [num_tokens * Hq][nsplit][D] (nsplit > 1)
  float* part_ml;             // [num_tokens * Hq][nsplit][2]
  int64_t page_stride, row_stride, head_stride, q_stride, out_stride, new_stride, table_stride;   // elements
  uint32_t page_magic, page_shift;   // j / page_size = j * magic >> shift for j < 2^31
  int32_t num_seqs, num_tokens, Hq, Hkv, group, page_size, num_pages, max_pages, max_seq_len, max_kv_len;
  int32_t window, sinks;
  float scale_log2;           // scale / ln 2
  int32_t row_tiles, nsplit, split_tiles;   // row tiles a sequence, splits, key tiles a split
};

constexpr int kPagedBlock = 256;
constexpr float kLn2 = 0.693147180559945309f;

struct PagedSeq {
  int start, q_len, first_pos;   // position of the first new token (negative: the first ones see nothing)
};

__device__ __forceinline__ PagedSeq paged_seq(const PagedArgs& a, int s) {
  PagedSeq q;
  int b = sload(a.seq_start + s), e = sload(a.seq_start + s + 1);
  b = b < 0 ? 0 : (b > a.num_tokens ? a.num_tokens : b);
  e = e < b ? b : (e > a.num_tokens ? a.num_tokens : e);
  q.start = b;
  q.q_len = e - b < a.max_seq_len ? e - b : a.max_seq_len;
  const int n = sload(a.kv_len + s);
  q.first_pos = (n < 0 ? 0 : n) - (e - b);
  return q;
}

__device__ __forceinline__ int page_of(const PagedArgs& a, int j) {
  return static_cast<int>((static_cast<uint64_t>(static_cast<uint32_t>(j)) * a.page_magic) >> a.page_shift);
}

// Page table entry of token j of sequence s (of its first token past the table's end).
__device__ __forceinline__ int page_entry(const PagedArgs& a, int s, int j) {
  const int pi = page_of(a, j);
  return gload(a.table + s * a.table_stride + (pi < a.max_pages ? pi : 0));
}

// Cache row of token j in elements (head 0), given its table entry; row 0 of the
// cache, and ok = false, when the token lies on no page or at or past `limit`.
__device__ __forceinline__ int64_t page_row(const PagedArgs& a, int page, int j, int limit, bool& ok) {
  const int pi = page_of(a, j);
  ok = (j < limit) & (pi < a.max_pages) & (page >= 0) & (page < a.num_pages);
  return ok ? page * a.page_stride + (j - pi * a.page_size) * a.row_stride : 0;
}

__device__ __forceinline__ int64_t cache_row(const PagedArgs& a, int s, int j, int limit, bool& ok) {
  return page_row(a, page_entry(a, s, j), j, limit, ok);
}

// Tiles of T keys that rows at positions [pmin, pmax] see: the first `sink`
// ones and those from `lo` to `hi`.
struct KeyTiles {
  int sink, lo, hi, count, limit;   // limit: first token no row sees
};

template <int T>
__device__ __forceinline__ KeyTiles key_tiles(const PagedArgs& a, int pmin, int pmax) {
  KeyTiles k;
  k.limit = pmax < a.max_kv_len ? pmax + 1 : a.max_kv_len;
  if (k.limit < 0) k.limit = 0;
  k.lo = 0;
  k.sink = 0;
  if (a.window > 0) {
    if (pmin >= a.window) {
      const int low = pmin - a.window + 1;
      k.sink = ((a.sinks < low ? a.sinks : low) + T - 1) / T;
      k.lo = low / T;
      if (k.lo < k.sink) k.lo = k.sink;
    }
  }
  k.hi = (k.limit + T - 1) / T;
  if (k.sink > k.hi) k.sink = k.hi;
  if (k.lo > k.hi) k.lo = k.hi;
  k.count = k.sink + (k.hi - k.lo);
  return k;
}

__device__ __forceinline__ int key_tile(const KeyTiles& k, int v) { return v < k.sink ? v : k.lo + (v - k.sink); }

// Bits set in each element of a raw word that is infinite or NaN (bit 15 and 31 for the
// 16-bit types, bit 31 for fp32).
template <int IT>
__device__ __forceinline__ uint32_t nonfinite_bits(uint32_t w) {
  if constexpr (IT == kBF16) return ((w & 0x7f807f80u) + 0x00800080u) & 0x80008000u;
  else if constexpr (IT == kF16) return ((w & 0x7c007c00u) + 0x04000400u) & 0x80008000u;
  else return ((w & 0x7f800000u) + 0x00800000u) & 0x80000000u;
}

template <int IT>
__device__ __forceinline__ bool nonfinite16(u32x4 v) {
  return (nonfinite_bits<IT>(v.x) | nonfinite_bits<IT>(v.y) | nonfinite_bits<IT>(v.z) | nonfinite_bits<IT>(v.w)) != 0;
}

// 16 raw bytes with every infinite or NaN element set to zero.
template <int IT>
__device__ __forceinline__ u32x4 finite16(u32x4 v) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t b = nonfinite_bits<IT>(v[i]);
    v[i] &= IT == kF32 ? (b != 0 ? 0u : ~0u) : ~((b >> 15) * 0xffffu);
  }
  return v;
}

// Scores of tokens a row may not see become -infinity.  bits: bit j where token
// j0 + j of the tile is on a page.
template <int JT>
__device__ __forceinline__ void mask_tile(const PagedArgs& a, f32x4 (&S)[JT], int j0, int pos, uint64_t bits, int g) {
  const int rel = pos - j0 - 4 * g;                       // o = j - j0 - 4g is visible up to here,
  const int low = a.window > 0 ? rel - a.window : -1;     // past here (o >= 0 > -1 without a window)
  const int sink = a.sinks - j0 - 4 * g;                  // or before here
#pragma unroll
  for (int jt = 0; jt < JT; ++jt) {
    const uint32_t on = static_cast<uint32_t>(bits >> (32 * (jt / 2))) >> (4 * g);
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int o = 16 * jt + r;
      const bool see = (o <= rel) & ((o > low) | (o < sink)) & ((on & (1u << (o & 31))) != 0);
      S[jt][r] = see ? S[jt][r] : -__builtin_inff();
    }
  }
}

// Running softmax of one row block (column li of each lane).
struct RowState {
  float m, l;   // reference point of the exponents (log2 units) and the lane's part of the sum
};

// The reference point follows the maximum only when it lags by more than 2^8:
// sums and products stay far from overflow, most tiles need no rescaling, and the exchange
// between lanes is left to the tiles that do.  fp16: the reference lies 2^7 below the maximum it was
// taken from, so that weights reach up to 2^15 and one below 2^-25 of the largest, of which a
// long cache may hold many, is not rounded to zero (2^-32 is; 2^-21 and more keep all their bits).
template <int IT>
constexpr float kBelow = IT == kF16 ? 7.0f : 0.0f;

template <int IT>
__device__ __forceinline__ bool lags(const PagedArgs& a, float mx, const RowState& st) {
  return mx * a.scale_log2 > st.m + (kBelow<IT> + 8.0f);
}

__device__ __forceinline__ float max4(float m, f32x4 v) {
  return fmaxf(fmaxf(fmaxf(m, v[0]), fmaxf(v[1], v[2])), v[3]);
}

// New reference point; the factor for the sum and the output so far.
template <int IT, int JT>
__device__ __forceinline__ float move_reference(const PagedArgs& a, const f32x4 (&S)[JT], RowState& st) {
  float mx = -__builtin_inff();
#pragma unroll
  for (int jt = 0; jt < JT; ++jt) mx = max4(mx, S[jt]);
  const float mn = fmaxf(st.m, max_groups(mx) * a.scale_log2 - kBelow<IT>);
  const float alpha = mn == st.m ? 1.0f : __builtin_amdgcn_exp2f(st.m - mn);
  st.m = mn;
  st.l *= alpha;
  return alpha;
}

// exp2(c S - m) of one D tile, added to `sum`, the lane's part of the key tile's sum (a running sum that
// took them one by one would lose weights below its last place).  Nothing visible so far: m is
// -infinity, and 0 in its place gives the weights exp2(-infinity) = 0.
__device__ __forceinline__ f32x4 weights(const PagedArgs& a, f32x4 S, float m, float& sum) {
  const float base = m == -__builtin_inff() ? 0.0f : m;
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    S[r] = __builtin_amdgcn_exp2f(fmaf(S[r], a.scale_log2, -base));
    sum += S[r];
  }
  return S;
}

// Store one row's results: the output, or this split's partial ones.
template <int IT, int DT>
__device__ __forceinline__ void store_row(const PagedArgs& a, const f32x4 (&O)[DT], float m, float l, int64_t token,
                                          int head, int split, int g) {
  typedef typename Mma<IT>::elem elem;
  if (a.nsplit == 1) {
    const float inv = l > 0.0f ? 1.0f / l : (l == 0.0f ? 0.0f : l);   // nothing visible: zeros; NaN stays
    elem* o = reinterpret_cast<elem*>(a.out) + token * a.out_stride + head * (DT * 16) + 4 * g;
#pragma unroll
    for (int d = 0; d < DT; ++d) narrow4<IT>(o + 16 * d, O[d] * inv);
    if (a.lse != nullptr && g == 0) a.lse[token * a.Hq + head] = (m + log2f(l)) * kLn2;
  } else {
    const int64_t at = (token * a.Hq + head) * a.nsplit + split;
    float* o = a.part_o + at * (DT * 16) + 4 * g;
#pragma unroll
    for (int d = 0; d < DT; ++d) *reinterpret_cast<f32x4*>(o + 16 * d) = O[d];
    if (g == 0) {
      a.part_ml[2 * at] = m;
      a.part_ml[2 * at + 1] = l;
    }
  }
}

__device__ __forceinline__ int64_t shfl64(int64_t v, int from) {
  const int lo = __shfl(static_cast<int>(v), from), hi = __shfl(static_cast<int>(v >> 32), from);
  return (static_cast<int64_t>(hi) << 32) | static_cast<uint32_t>(lo);
}

template <int IT, int D, int RB>
__global__ __launch_bounds__(kPagedBlock, IT == kF32 ? 1 : 2) void paged_tile_kernel(PagedArgs a) {
  typedef typename Mma<IT>::elem elem;
  typedef typename Mma<IT>::frag frag;
  constexpr int T = 64, JT = T / 16, KS = D / 32, DT = D / 16;
  constexpr int kVec = 16 / sizeof(elem), kPerRow = D / kVec, kRowsPass = kPagedBlock / kPerRow, kPasses = T / kRowsPass;
  constexpr int kPitch = tile_pitch<IT>(D);
  constexpr int kRows = 64 * RB;
  __shared__ __align__(16) elem lds[2][2][T * kPitch];   // [buffer][K, V]
  __shared__ int64_t rows_at[4][T];   // cache rows (elements) of a tile's tokens (tile v in slot v mod 4),
  __shared__ uint64_t on_pages[4];    // and which of them lie on a page
  __shared__ int odd;                 // an output is infinite or NaN
  const int tid = threadIdx.x, lane = tid & 63, g = lane >> 4, li = lane & 15;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  int item = xcd_order(blockIdx.x, gridDim.x);
  const int split = item % a.nsplit;
  item /= a.nsplit;
  const int rt = a.row_tiles - 1 - item % a.row_tiles;   // later tokens see more keys: first
  item /= a.row_tiles;
  const int kvh = item % a.Hkv, s = item / a.Hkv;
  const PagedSeq sq = paged_seq(a, s);
  const int total_rows = sq.q_len * a.group, row0 = rt * kRows;
  if (row0 >= total_rows) return;
  const int row1 = row0 + kRows < total_rows ? row0 + kRows : total_rows;
  const KeyTiles kt = key_tiles<T>(a, sq.first_pos + row0 / a.group, sq.first_pos + (row1 - 1) / a.group);
  const int v0 = split * a.split_tiles;
  const int v1 = split == a.nsplit - 1 || kt.count - v0 < a.split_tiles ? kt.count : v0 + a.split_tiles;

  frag Q[RB][KS];
  int pos[RB], head[RB];
  int64_t tok[RB];
#pragma unroll
  for (int b = 0; b < RB; ++b) {
    const int R = row0 + (wave * RB + b) * 16 + li;
    const bool in = R < row1;
    const int t = in ? R / a.group : 0;
    tok[b] = in ? sq.start + t : -1;
    head[b] = kvh * a.group + (in ? R - t * a.group : 0);
    pos[b] = in && sq.first_pos + t >= 0 ? sq.first_pos + t : -1;
    const elem* qp = reinterpret_cast<const elem*>(a.q) + (in ? tok[b] : sq.start) * a.q_stride + static_cast<int64_t>(head[b]) * D + 8 * g;
#pragma unroll
    for (int k = 0; k < KS; ++k) Q[b][k] = frag_row<IT>(qp + 32 * k);
  }
  // positions of the wavefront's rows (uniform)
  const int w0 = row0 + wave * RB * 16, w1 = w0 + RB * 16 < row1 ? w0 + RB * 16 : row1;
  const int wmin = w1 == w0 + RB * 16 ? sq.first_pos + w0 / a.group : -1;   // -1: some rows see nothing
  const int wmax = w0 < w1 ? sq.first_pos + (w1 - 1) / a.group : -1;

  f32x4 O[RB][DT];
  RowState rs[RB];
  const int64_t hoff = static_cast<int64_t>(kvh) * a.head_stride;
  const int vec = tid % kPerRow, srow = tid / kPerRow;
  const char* const kbase = a.k + (hoff + vec * kVec) * static_cast<int64_t>(sizeof(elem));
  const char* const vbase = a.v + (hoff + vec * kVec) * static_cast<int64_t>(sizeof(elem));
  // Tokens that no row may see are read from row 0: their weights are zero.
  u32x4 kr[kPasses], vr[kPasses];
  auto fetch = [&](int slot) {
#pragma unroll
    for (int i = 0; i < kPasses; ++i) {
      const int64_t at = rows_at[slot][srow + i * kRowsPass] * static_cast<int64_t>(sizeof(elem));
      kr[i] = ld<false, u32x4>(kbase + at);
      vr[i] = ld<false, u32x4>(vbase + at);
    }
  };
  // An infinite or NaN element of V would reach rows that may not see it (0 times it is
  // not 0).  The tiles run as if there were none; when an output came out infinite or NaN they
  // run once more with zeros for such elements, and a last pass gives them to the rows that
  // see them.
  bool clean = false;
  auto put = [&](int buf) {
    if (__builtin_expect(clean, 0)) {
#pragma unroll
      for (int i = 0; i < kPasses; ++i) vr[i] = finite16<IT>(vr[i]);
    }
#pragma unroll
    for (int i = 0; i < kPasses; ++i) {
      const int at = (srow + i * kRowsPass) * kPitch + vec * kVec;
      *reinterpret_cast<u32x4*>(&lds[buf][0][at]) = kr[i];
      *reinterpret_cast<u32x4*>(&lds[buf][1][at]) = vr[i];
    }
  };
  // The page table is read by one wavefront a tile, in turn, two tiles ahead: `entry` is requested
  // a tile before page_rows turns it into cache rows (loads complete in order, so it must not
  // be looked at while keys that were requested before it are in flight).
  int entry = 0;
  auto page_rows = [&](int v) {
    bool ok;
    const int64_t row = page_row(a, entry, key_tile(kt, v) * T + lane, kt.limit, ok);
    rows_at[(v - v0) & 3][lane] = row;
    const uint64_t bits = __ballot(ok);
    if (lane == 0) on_pages[(v - v0) & 3] = bits;
  };
  auto turn = [&](int v) { return ((v - v0) & 3) == wave && v < v1; };
  f32x4 S[RB][JT];
  bool work = false;
  uint64_t on_page = 0;
  // first half of a tile: scores, masks, reference points
  auto scores = [&](int v) {
    const int j0 = key_tile(kt, v) * T;
    work = j0 <= wmax;
    if (!work) return;
    const elem* Kt = lds[(v - v0) & 1][0];
    const bool full = on_page == ~0ull && j0 + T - 1 <= wmin &&
                      (a.window == 0 || j0 > wmax - a.window || j0 + T <= a.sinks);
    // the next 16 keys' fragments are read while the matrix cores take the current ones
    frag kf[2][KS];
#pragma unroll
    for (int k = 0; k < KS; ++k) kf[0][k] = frag_row<IT>(Kt + li * kPitch + 32 * k + 8 * g);
#pragma unroll
    for (int jt = 0; jt < JT; ++jt) {
      if (jt + 1 < JT) {
#pragma unroll
        for (int k = 0; k < KS; ++k) kf[(jt + 1) & 1][k] = frag_row<IT>(Kt + (16 * (jt + 1) + li) * kPitch + 32 * k + 8 * g);
      }
#pragma unroll
      for (int b = 0; b < RB; ++b) S[b][jt] = f32x4{0, 0, 0, 0};
#pragma unroll
      for (int k = 0; k < KS; ++k)
#pragma unroll
        for (int b = 0; b < RB; ++b) S[b][jt] = mma<IT>(kf[jt & 1][k], Q[b][k], S[b][jt]);
      __builtin_amdgcn_sched_barrier(0);
    }
    if (!full) {
      asm volatile("");   // a branch, not 200 selects in every tile
#pragma unroll
      for (int b = 0; b < RB; ++b) mask_tile<JT>(a, S[b], j0, pos[b], on_page, g);
    }
    bool move = false;
#pragma unroll
    for (int b = 0; b < RB; ++b) {
      float mx = -__builtin_inff();
#pragma unroll
      for (int jt = 0; jt < JT; ++jt) mx = max4(mx, S[b][jt]);
      move |= lags<IT>(a, mx, rs[b]);
    }
    if (__ballot(move) != 0) {
#pragma unroll
      for (int b = 0; b < RB; ++b) {
        const float alpha = move_reference<IT, JT>(a, S[b], rs[b]);
#pragma unroll
        for (int d = 0; d < DT; ++d) O[b][d] *= alpha;
      }
    }
  };
  // second half: weights, output
  auto outputs = [&](int v) {
    if (!work) return;
    const elem* Vt = lds[(v - v0) & 1][1];
    float sum[RB];
#pragma unroll
    for (int b = 0; b < RB; ++b) sum[b] = 0.0f;
#pragma unroll
    for (int h = 0; h < JT / 2; ++h) {
      // rounded once: a second part, as single tokens have it, would repeat this product, 18% of the kernel
      // (error against 64 bits 0.0023 instead of the plain form's 0.0017 in bf16, 0.00029 and 0.00021 in fp16)
      frag P[RB];
#pragma unroll
      for (int b = 0; b < RB; ++b)
        P[b] = to_frag<IT>(stack(weights(a, S[b][2 * h], rs[b].m, sum[b]), weights(a, S[b][2 * h + 1], rs[b].m, sum[b])));
#pragma unroll
      for (int d = 0; d < DT; ++d) {
        const frag vf = frag_col<IT>(Vt, kPitch, 32 * h, 16 * d, lane);
#pragma unroll
        for (int b = 0; b < RB; ++b) O[b][d] = mma<IT>(vf, P[b], O[b][d]);
      }
    }
#pragma unroll
    for (int b = 0; b < RB; ++b) rs[b].l += sum[b];
  };
  if (tid == 0) odd = 0;
  for (;;) {
#pragma unroll
    for (int b = 0; b < RB; ++b) {
      rs[b].m = -__builtin_inff();
      rs[b].l = 0.0f;
#pragma unroll
      for (int d = 0; d < DT; ++d) O[b][d] = f32x4{0, 0, 0, 0};
    }
    for (int v = v0; v < v0 + 3; ++v)
      if (turn(v)) entry = page_entry(a, s, key_tile(kt, v) * T + lane);
    if (turn(v0)) page_rows(v0);
    if (turn(v0 + 1)) page_rows(v0 + 1);
    __syncthreads();
    if (v0 < v1) {
      fetch(0);
      put(0);
    }
    __syncthreads();
    for (int v = v0; v < v1; ++v) {
      const uint64_t bits = on_pages[(v - v0) & 3];
      on_page = (static_cast<uint64_t>(static_cast<uint32_t>(__builtin_amdgcn_readfirstlane(static_cast<int>(bits >> 32)))) << 32) |
                static_cast<uint32_t>(__builtin_amdgcn_readfirstlane(static_cast<int>(bits)));
      if (turn(v + 3)) entry = page_entry(a, s, key_tile(kt, v + 3) * T + lane);
      if (v + 1 < v1) fetch((v + 1 - v0) & 3);
      scores(v);
      outputs(v);
      if (v + 1 < v1) put((v + 1 - v0) & 1);
      if (turn(v + 2)) page_rows(v + 2);   // over tile v - 2's, which no wavefront reads any more
      __syncthreads();
    }
    if (clean) break;
    float any = 0.0f;
#pragma unroll
    for (int b = 0; b < RB; ++b)
#pragma unroll
      for (int d = 0; d < DT; ++d) any += (O[b][d][0] + O[b][d][1]) + (O[b][d][2] + O[b][d][3]);
    if (__ballot(!(fabsf(any) < __builtin_inff())) != 0) odd = 1;
    __syncthreads();
    if (__builtin_expect(odd == 0, 1)) break;
    clean = true;
  }
  if (__builtin_expect(clean, 0)) {
    // rare: the tiles once more from the cache, for the infinities and NaN among the values of
    // tokens that a row sees (its weight is not zero)
#pragma unroll 1
    for (int v = v0; v < v1; ++v) {
      const int j0 = key_tile(kt, v) * T;
      bool there, any = false;
      const int64_t row = cache_row(a, s, j0 + lane, kt.limit, there);
      const uint64_t bits = __ballot(there);
      const elem* base = reinterpret_cast<const elem*>(a.v) + row + hoff;
      for (int i = 0; i < kPerRow; ++i) any |= nonfinite16<IT>(*reinterpret_cast<const u32x4*>(base + i * kVec));
      if (j0 > wmax || __ballot(any) == 0) continue;
#pragma unroll 1
      for (int h = 0; h < JT / 2; ++h) {
        frag P[RB];
#pragma unroll
        for (int b = 0; b < RB; ++b) {
          f32x4 sc[JT];
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            const elem* kp = reinterpret_cast<const elem*>(a.k) + shfl64(row, 32 * h + 16 * u + li) + hoff + 8 * g;
            sc[u] = f32x4{0, 0, 0, 0};
#pragma unroll
            for (int k = 0; k < KS; ++k) sc[u] = mma<IT>(frag_row<IT>(kp + 32 * k), Q[b][k], sc[u]);
            sc[u + 2] = sc[u];
          }
          mask_tile<JT>(a, sc, j0 + 32 * h, pos[b], bits >> (32 * h), g);
          float unused = 0.0f;
          P[b] = to_frag<IT>(stack(weights(a, sc[0], rs[b].m, unused), weights(a, sc[1], rs[b].m, unused)));
        }
#pragma unroll
        for (int d = 0; d < DT; ++d) {
          f32x8 x;
#pragma unroll
          for (int e = 0; e < 8; ++e)
            x[e] = elem_to_float<IT>((reinterpret_cast<const elem*>(a.v) + hoff + li)[shfl64(row, 32 * h + 16 * (e >> 2) + 4 * g + (e & 3)) + 16 * d]);
#pragma unroll
          for (int b = 0; b < RB; ++b) O[b][d] = add_odd<IT>(x, P[b], O[b][d]);
        }
      }
    }
  }
#pragma unroll
  for (int b = 0; b < RB; ++b) {
    const float l = sum_groups(rs[b].l);
    if (tok[b] >= 0) store_row<IT, DT>(a, O[b], rs[b].m, l, tok[b], head[b], split, g);
  }
}

template <int IT, int D>
__global__ __launch_bounds__(kPagedBlock, IT == kF32 ? 1 : 2) void paged_row_kernel(PagedArgs a) {
  typedef typename Mma<IT>::elem elem;
  typedef typename Mma<IT>::frag frag;
  constexpr int T = 32, JT = 2, KS = D / 32, DT = D / 16, W = kPagedBlock / 64;
  constexpr int kVec = 16 / sizeof(elem), kPerRow = D / kVec, kRowsPass = 64 / kPerRow, kPasses = T / kRowsPass;
  constexpr int kPitch = tile_pitch<IT>(D);
  constexpr int kTileBytes = W * T * kPitch * sizeof(elem), kJoinBytes = W * 16 * (D + 4) * 4;
  __shared__ __align__(16) char lds[kTileBytes > kJoinBytes ? kTileBytes : kJoinBytes];
  __shared__ float jm[W][16], jl[W][16];
  const int tid = threadIdx.x, lane = tid & 63, g = lane >> 4, li = lane & 15;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  int item = xcd_order(blockIdx.x, gridDim.x);
  // heads first: workgroups that run together read neighbouring rows of the same pages
  const int kvh = item % a.Hkv;
  item /= a.Hkv;
  const int split = item % a.nsplit, s = item / a.nsplit;
  const PagedSeq sq = paged_seq(a, s);
  const int rows = sq.q_len * a.group;
  if (rows == 0) return;
  const KeyTiles kt = key_tiles<T>(a, sq.first_pos, sq.first_pos + sq.q_len - 1);
  const int v0 = split * a.split_tiles;
  const int v1 = split == a.nsplit - 1 || kt.count - v0 < a.split_tiles ? kt.count : v0 + a.split_tiles;
  const bool in = li < rows;
  const int t = in ? li / a.group : 0;
  const int64_t tok = sq.start + t;
  const int head = kvh * a.group + (in ? li - t * a.group : 0);
  const int pos = in && sq.first_pos + t >= 0 ? sq.first_pos + t : -1;
  frag Q[KS];
  {
    const elem* qp = reinterpret_cast<const elem*>(a.q) + tok * a.q_stride + static_cast<int64_t>(head) * D + 8 * g;
#pragma unroll
    for (int k = 0; k < KS; ++k) Q[k] = frag_row<IT>(qp + 32 * k);
  }
  f32x4 O[DT];
#pragma unroll
  for (int d = 0; d < DT; ++d) O[d] = f32x4{0, 0, 0, 0};
  RowState rs{-__builtin_inff(), 0.0f};
  elem* const Vt = reinterpret_cast<elem*>(lds) + wave * T * kPitch;
  const int64_t hoff = static_cast<int64_t>(kvh) * a.head_stride;
  const int vec = lane % kPerRow, srow = lane / kPerRow;
  u32x4 kr[JT][KS * sizeof(elem) / 2], vr[kPasses];
  auto fetch = [&](int64_t row_off) {   // lane l holds the cache row of token l % 32
#pragma unroll
    for (int jt = 0; jt < JT; ++jt) {
      const char* p = a.k + (shfl64(row_off, 16 * jt + li) + hoff + 8 * g) * static_cast<int64_t>(sizeof(elem));
#pragma unroll
      for (int k = 0; k < KS; ++k) {
        if constexpr (IT == kF32) {
          kr[jt][2 * k] = ld<false, u32x4>(p + 128 * k);
          kr[jt][2 * k + 1] = ld<false, u32x4>(p + 128 * k + 16);
        } else {
          kr[jt][k] = ld<false, u32x4>(p + 64 * k);
        }
      }
    }
#pragma unroll
    for (int i = 0; i < kPasses; ++i)
      vr[i] = ld<true, u32x4>(a.v + (shfl64(row_off, srow + i * kRowsPass) + hoff + vec * kVec) * static_cast<int64_t>(sizeof(elem)));
  };
  const int first = v0 + wave;
  int entry = 0;
  bool ok = false;
  if (first < v1) {
    const int64_t off = cache_row(a, s, key_tile(kt, first) * T + (lane & 31), kt.limit, ok);
    if (first + W < v1) entry = page_entry(a, s, key_tile(kt, first + W) * T + (lane & 31));
    fetch(off);
  }
  for (int v = first; v < v1; v += W) {
    const int j0 = key_tile(kt, v) * T;
    const uint64_t on_page = __ballot(ok) & 0xffffffffull;
    bool bad = false;
    frag K[JT][KS];
#pragma unroll
    for (int jt = 0; jt < JT; ++jt)
#pragma unroll
      for (int k = 0; k < KS; ++k) {
        if constexpr (IT == kF32) {
          const u32x4 u = kr[jt][2 * k], w = kr[jt][2 * k + 1];
          K[jt][k] = __builtin_bit_cast(frag, u32x8{u.x, u.y, u.z, u.w, w.x, w.y, w.z, w.w});
        } else {
          K[jt][k] = __builtin_bit_cast(frag, kr[jt][k]);
        }
      }
    f32x4 S[JT];
#pragma unroll
    for (int jt = 0; jt < JT; ++jt) {
      S[jt] = f32x4{0, 0, 0, 0};
#pragma unroll
      for (int k = 0; k < KS; ++k) S[jt] = mma<IT>(K[jt][k], Q[k], S[jt]);
    }
#pragma unroll
    for (int i = 0; i < kPasses; ++i) {
      bad |= nonfinite16<IT>(vr[i]);
      *reinterpret_cast<u32x4*>(Vt + (srow + i * kRowsPass) * kPitch + vec * kVec) = vr[i];
    }
    bad = __ballot(bad) != 0;
    if (v + W < v1) {   // (loads complete in order: entries before the keys, looked at a tile later)
      const int64_t off = page_row(a, entry, key_tile(kt, v + W) * T + (lane & 31), kt.limit, ok);
      if (v + 2 * W < v1) entry = page_entry(a, s, key_tile(kt, v + 2 * W) * T + (lane & 31));
      fetch(off);
    }
    mask_tile<JT>(a, S, j0, pos, on_page, g);
    if (__ballot(lags<IT>(a, max4(max4(-__builtin_inff(), S[0]), S[1]), rs)) != 0) {
      const float alpha = move_reference<IT, JT>(a, S, rs);
#pragma unroll
      for (int d = 0; d < DT; ++d) O[d] *= alpha;
    }
    float sum = 0.0f;
    S[0] = weights(a, S[0], rs.m, sum);
    S[1] = weights(a, S[1], rs.m, sum);
    rs.l += sum;
    __builtin_amdgcn_wave_barrier();
    // the matrix cores idle beside the cache's stream: the weights go through in two
    // parts (16 bits and more; fp16 within 2^-32 of the row's largest weight), so that the
    // output's rounding is the one that counts
    const f32x8 w = stack(S[0], S[1]);
    const frag P = to_frag<IT>(w);
    frag P1;
    if constexpr (IT != kF32) P1 = to_frag<IT>(w - from_frag<IT>(P));
    if (__builtin_expect(bad, 0)) {
      // the same products over the finite values, so that one that no query sees changes no bit
#pragma unroll
      for (int d = 0; d < DT; ++d) {
        const f32x8 x = from_frag<IT>(frag_col<IT>(Vt, kPitch, 0, 16 * d, lane));
        if constexpr (IT != kF32) O[d] = mma<IT>(finite_part<IT>(x), P1, O[d]);
        O[d] = add_odd<IT>(x, P, mma<IT>(finite_part<IT>(x), P, O[d]));
      }
    } else {
#pragma unroll
      for (int d = 0; d < DT; ++d) {
        const frag vf = frag_col<IT>(Vt, kPitch, 0, 16 * d, lane);
        if constexpr (IT != kF32) O[d] = mma<IT>(vf, P1, O[d]);
        O[d] = mma<IT>(vf, P, O[d]);
      }
    }
    __builtin_amdgcn_wave_barrier();
  }
  // join the four wavefronts
  __syncthreads();
  float* const jo = reinterpret_cast<float*>(lds);   // [W][16][D + 4]
  const float l = sum_groups(rs.l);
  if (g == 0) {
    jm[wave][li] = rs.m;
    jl[wave][li] = l;
  }
#pragma unroll
  for (int d = 0; d < DT; ++d) *reinterpret_cast<f32x4*>(jo + (wave * 16 + li) * (D + 4) + 16 * d + 4 * g) = O[d];
  __syncthreads();
  if (wave == 0) {
    float m = jm[0][li];
#pragma unroll
    for (int w = 1; w < W; ++w) m = fmaxf(m, jm[w][li]);
    const float base = m == -__builtin_inff() ? 0.0f : m;
    float sum = 0.0f;
#pragma unroll
    for (int d = 0; d < DT; ++d) O[d] = f32x4{0, 0, 0, 0};
#pragma unroll
    for (int w = 0; w < W; ++w) {
      const float f = __builtin_amdgcn_exp2f(jm[w][li] - base);
      sum += jl[w][li] * f;
#pragma unroll
      for (int d = 0; d < DT; ++d) O[d] += *reinterpret_cast<const f32x4*>(jo + (w * 16 + li) * (D + 4) + 16 * d + 4 * g) * f;
    }
    if (in) store_row<IT, DT>(a, O, m, sum, tok, head, split, g);
  }
}

// Joins the splits of a (token, head), eight partial outputs in flight, lanes over
// head_dim.  kShare: the workgroup's wavefronts share the splits of one row (many
// splits); otherwise each takes a row of its own.  Maxima leave NaN out, so the weight of a
// split whose scores are all NaN is zero: its NaN reaches the row through the sum.
template <int IT, int D, bool kShare>
__global__ __launch_bounds__(kPagedBlock) void paged_join_kernel(PagedArgs a) {
  typedef typename Mma<IT>::elem elem;
  constexpr int E = D / 64, W = kPagedBlock / 64, U = 8;
  __shared__ float jo[W][D], jl[W];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t row = kShare ? blockIdx.x : static_cast<int64_t>(blockIdx.x) * W + wave;
  const int64_t token = row / a.Hq;
  if (token >= a.num_tokens) return;
  // rows that belong to no sequence were not computed: leave them alone
  int lo = 0, hi = a.num_seqs;
  while (lo < hi) {   // first sequence whose end lies past the token
    const int mid = (lo + hi) >> 1;
    if (sload(a.seq_start + mid + 1) > token) hi = mid;
    else lo = mid + 1;
  }
  if (lo >= a.num_seqs) return;
  const PagedSeq sq = paged_seq(a, lo);
  if (token < sq.start || token - sq.start >= sq.q_len) return;
  const int head = static_cast<int>(row - token * a.Hq);
  const float* ml = a.part_ml + row * a.nsplit * 2;
  const float* po = a.part_o + row * a.nsplit * D + lane * E;
  float m = -__builtin_inff();
  for (int k = lane; k < a.nsplit; k += 64) m = fmaxf(m, ml[2 * k]);
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) m = fmaxf(m, __shfl_xor(m, d));
  const float base = m == -__builtin_inff() ? 0.0f : m;
  float l = 0.0f, o[E];
#pragma unroll
  for (int e = 0; e < E; ++e) o[e] = 0.0f;
  for (int k0 = kShare ? wave * U : 0; k0 < a.nsplit; k0 += kShare ? W * U : U) {
    float p[U][E], w[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int k = k0 + u < a.nsplit ? k0 + u : a.nsplit - 1;
      w[u] = k0 + u < a.nsplit ? __builtin_amdgcn_exp2f(ml[2 * k] - base) : 0.0f;
      l = fmaf(ml[2 * k + 1], w[u], l);   // the sum of a split with a NaN score is NaN, whatever its weight
#pragma unroll
      for (int e = 0; e < E; ++e) p[u][e] = po[static_cast<int64_t>(k) * D + e];
    }
#pragma unroll
    for (int u = 0; u < U; ++u)   // a weight of zero hides an infinity or NaN among the split's values
#pragma unroll
      for (int e = 0; e < E; ++e) o[e] = w[u] != 0.0f ? fmaf(p[u][e], w[u], o[e]) : o[e];
  }
  elem* out = reinterpret_cast<elem*>(a.out) + token * a.out_stride + static_cast<int64_t>(head) * D;
  auto store = [&](int d, float v) {
    if constexpr (IT == kF32) out[d] = v;
    else if constexpr (IT == kBF16) out[d] = __builtin_bit_cast(uint16_t, static_cast<__bf16>(v));
    else out[d] = __builtin_bit_cast(uint16_t, static_cast<_Float16>(v));
  };
  const int d = threadIdx.x;
  if constexpr (kShare) {
#pragma unroll
    for (int e = 0; e < E; ++e) jo[wave][lane * E + e] = o[e];
    if (lane == 0) jl[wave] = l;
    __syncthreads();
    l = (jl[0] + jl[1]) + (jl[2] + jl[3]);
  }
  const float inv = l > 0.0f ? 1.0f / l : (l == 0.0f ? 0.0f : l);
  if constexpr (kShare) {
    if (d < D) store(d, ((jo[0][d] + jo[1][d]) + (jo[2][d] + jo[3][d])) * inv);
  } else {
#pragma unroll
    for (int e = 0; e < E; ++e) store(lane * E + e, o[e] * inv);
  }
  if (a.lse != nullptr && (kShare ? d : lane) == 0) a.lse[token * a.Hq + head] = (m + log2f(l)) * kLn2;
}

// Append: one thread a 16-byte vector of one new token's keys and values.
template <int ES>
__global__ __launch_bounds__(kPagedBlock) void paged_append_kernel(PagedArgs a, int head_vecs) {
  const int per = a.Hkv * head_vecs;
  const int64_t at = static_cast<int64_t>(blockIdx.x) * kPagedBlock + threadIdx.x;
  const int64_t token = at / per;
  if (token >= a.num_tokens) return;
  const int v = static_cast<int>(at - token * per), h = v / head_vecs;
  int lo = 0, hi = a.num_seqs;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (gload(a.seq_start + mid + 1) > token) hi = mid;
    else lo = mid + 1;
  }
  if (lo >= a.num_seqs) return;
  const int start = gload(a.seq_start + lo), end = gload(a.seq_start + lo + 1);
  if (token < start) return;
  const int64_t j = static_cast<int64_t>(gload(a.kv_len + lo)) - (end < a.num_tokens ? end : a.num_tokens) + token;
  if (j < 0 || j > INT32_MAX - 1) return;
  bool ok;
  const int64_t row = cache_row(a, lo, static_cast<int>(j), INT32_MAX, ok);
  if (!ok) return;
  const int64_t src = (token * a.new_stride) * ES + v * 16;
  const int64_t dst = (row + h * a.head_stride) * ES + (v - h * head_vecs) * 16;
  st<false>(a.k + dst, ld<false, u32x4>(a.k_new + src));
  st<false>(a.v + dst, ld<false, u32x4>(a.v_new + src));
}

}  // namespace rssm
