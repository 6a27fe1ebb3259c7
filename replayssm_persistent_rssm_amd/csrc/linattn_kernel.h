// linattn_kernel.h -- gfx950 kernels of linear attention with a decay for each
// head: the chunked prompt form and the single-token form.
//
// A chunk of Q = 64 tokens with l_i = sum_{u <= i} dt_u A inside it and starting
// state S0 gives
//     y_i = exp(l_i) S0 C_i + sum_{j <= i} exp(l_i - l_j) dt_j (C_i . B_j) x_j + D x_i
//     S'  = exp(l_Q) S0 + sum_j w_j x_j B_j^T,    w_j = exp(l_Q - l_j) dt_j.
// One workgroup of 4 wavefronts holds one 64-row tile of one head's state in
// registers and walks the chunks of one stretch of one sequence.  Everything
// is laid out transposed, so that each product's D tiles are the next one's operand
// (mma_device.h):
//   scores  G^T[j][i] = B_j . C_i          A = B rows (LDS), Bm = C rows (global -> registers)
//   y^T[p][i] = S0[p] . C_i                A = S0 rows (LDS, rounded), Bm = the same C rows
//       times exp(l_i), a scalar of the lane's column i
//   y^T += x^T M^T                         A = x columns (LDS), Bm = masked weighted scores
//   S'^T[n][p] = B^T (w x)                 A = B columns (LDS), Bm = w_j x_j in parts of the
//                                          input type (fp16: scaled by powers of two)
// Wavefront w owns tokens 16w .. 16w+15 of y and state rows 16w .. 16w+15 of the
// update.  The next chunk's inputs are loaded into registers while the current
// one is computed.  A chunk of 64 keeps two workgroups a compute unit (57 KiB of LDS
// and 201 registers for bf16); a third (168 registers) ran no faster.
//
// When sequences x heads are too few to fill the chip, the token axis is split into
// stretches: one launch folds each stretch from a zero state (kStateOnly), a second scans the
// stretches' states and decays, a third computes the outputs from the
// scanned starting states.
//
// Bound by the vector ALUs and LDS together: two wavefronts a SIMD do not fill either.  12 ragged prompts,
// 13,649 tokens, 256 heads in 8 groups, gated, fp32 state: 0.58 ms, 2.7 TB/s of the bytes it cannot do without
// (0.60 ms with z and y in 8-byte pieces); 466 vector, 88 matrix and 111 LDS instructions a wavefront and chunk keep
// the vector ALUs busy 44% of the time, LDS 48% (and 10% more in bank conflicts), the matrix cores 26%.  Of that time, the gate takes 13%, three quarters of the score and
// starting-state products 13%, two of the three parts of the state update 6% (each timed by leaving it
// out).  One prompt of 16,384 tokens, 64 heads, bf16 state, in 8 stretches: 0.22 ms, a quarter of it the
// fold.
#pragma once

#include "mma_device.h"

namespace rssm {

struct LinArgs {
  char* state;
  const float* A;
  const float* D;         // [H] or null
  const float* dt_bias;   // [H] or null
  const char* x;
  const char* B;
  const char* C;
  const float* dt;        // or null
  const char* z;          // or null
  char* y;
  const int32_t* slots;
  const int32_t* seq_start;
  const int32_t* load_state;   // or null
  float* ws_state;        // [seqs][nseg][H][dim][dstate] (nseg > 1)
  float* ws_decay;        // [seqs][nseg][H] log decay of each stretch
  int64_t state_stride, x_stride, B_stride, C_stride, dt_stride, z_stride, y_stride;   // elements
  int32_t num_seqs, num_tokens, H, hpg, dim, num_slots, pad, max_seq_len, dt_softplus;
  int32_t nseg, seg_len;  // stretches of the token axis and their length (a multiple of 64)
};

// State row of row m of D tile p of y^T: the four rows that a lane group holds of tiles 2k and
// 2k + 1 are 8 consecutive ones, 16 bytes of z and y.
__device__ __forceinline__ constexpr int row_of(int p, int m) { return 32 * (p >> 1) + 4 * (p & 1) + 8 * (m >> 2) + (m & 3); }

constexpr int kLinQ = 64;       // tokens a chunk
constexpr int kLinP = 64;       // state rows a workgroup
constexpr int kLinBlock = 256;

// Sequence s of the call: slot, first row and length, after the guards.
struct LinSeq {
  int slot, start, len;
  bool live;
};

__device__ __forceinline__ LinSeq lin_seq(const LinArgs& a, int s) {
  LinSeq q;
  q.slot = sload(a.slots + s);
  q.live = q.slot != a.pad && q.slot >= 0 && q.slot < a.num_slots;
  int b = sload(a.seq_start + s), e = sload(a.seq_start + s + 1);
  b = b < 0 ? 0 : (b > a.num_tokens ? a.num_tokens : b);
  e = e < b ? b : (e > a.num_tokens ? a.num_tokens : e);
  q.start = b;
  q.len = e - b < a.max_seq_len ? e - b : a.max_seq_len;
  return q;
}

template <int ST>
__device__ __forceinline__ f32x4 load_state4(const char* p) {
  return widen4<ST>(reinterpret_cast<const typename Mma<ST>::elem*>(p));
}
template <int ST>
__device__ __forceinline__ void store_state4(char* p, f32x4 v) {
  narrow4<ST>(reinterpret_cast<typename Mma<ST>::elem*>(p), v);
}

// 2^k by exponent bits, k in [-126, 127].
__device__ __forceinline__ float pow2i(int k) { return __uint_as_float(static_cast<uint32_t>(k + 127) << 23); }

// Exponent k such that 2^k brings a magnitude m (finite, >= 0) into [2^top,
// 2^(top + 1)); 0 for m = 0 or non-finite m.  At most 60, so that 2^k times fp32 sums stays finite.
__device__ __forceinline__ int scale_exp(float m, int top) {
  const int e = static_cast<int>(__float_as_uint(m) >> 23) - 127;
  if (!(m > 0.0f) || e == 128) return 0;
  const int k = top - e;
  return k > 60 ? 60 : (k < -110 ? -110 : k);
}

template <int IT, int N>
struct LinLds {
  typedef typename Mma<IT>::elem elem;
  static constexpr int kN = tile_pitch<IT>(N);
  static constexpr int kP = tile_pitch<IT>(kLinP);
  static constexpr int kS = N + 16 / static_cast<int>(sizeof(elem));   // read by rows only: rows 4 banks apart
  alignas(16) elem Bs[kLinQ * kN];
  alignas(16) elem Ss[kLinP * kS];
  alignas(16) elem Xs[kLinQ * kP];
  // four chunks at a time: l_i in log2 units from the end of the 16 tokens before i's
  // tile, exp(l_i), dt_i, w_i, and for tiles 1 .. 3 the weight exp(l_ref - l_j) dt_j of an
  // earlier token up to the tile's start (both factors of exp(l_i - l_j) then shrink
  // where the decay does, and only the tile on the diagonal needs one exponential a pair)
  alignas(16) float lr[4][kLinQ], e[4][kLinQ], dt[4][kLinQ], w[4][kLinQ], before[4][3][kLinQ];
  // for the diagonal, in log2 units: dt_i A, and its sum from the start of i's group of 4 tokens
  // (k = 0), of the group before (1) and of the one before that (2) up to i
  alignas(16) float da[4][kLinQ], since[4][3][kLinQ];
  // the whole chunk's decay and its logarithm
  float decay[4], total[4];
  alignas(16) float sinv[kLinP];   // fp16: inverse scale of each state row in Ss
};

// Stages 64 rows of COLS elements through registers, rows past the sequence as
// zeros: the buffer size ends with its last row.
template <int IT, int COLS>
struct Stage {
  typedef typename Mma<IT>::elem elem;
  static constexpr int kVec = 16 / sizeof(elem);
  static constexpr int kPerRow = COLS / kVec;
  static constexpr int kN = kLinQ * kPerRow / kLinBlock;
  u32x4 v[kN];
  uint32_t at[kN];
  __device__ __forceinline__ void init(uint32_t row_bytes, int tid) {
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      const int k = tid + i * kLinBlock;
      at[i] = (k / kPerRow) * row_bytes + (k % kPerRow) * 16;
    }
  }
  __device__ __forceinline__ void load(const char* base, uint32_t row_bytes, int rows) {
    const rsrc_t r = make_rsrc(base, (rows - 1) * row_bytes + COLS * sizeof(elem));
#pragma unroll
    for (int i = 0; i < kN; ++i) v[i] = bload16<false>(r, at[i], 0);
  }
  __device__ __forceinline__ void store(elem* tile, int pitch, int tid) const {
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      const int k = tid + i * kLinBlock;
      *reinterpret_cast<u32x4*>(tile + (k / kPerRow) * pitch + (k % kPerRow) * kVec) = v[i];
    }
  }
};

// exp(x) from the hardware's exp2: the product x log2(e) is carried in two parts, so that
// the result is within a few units of the last place at any x.
__device__ __forceinline__ float exp_near(float x) {
  const float y = x * 1.44269502f;                              // log2(e) = 1.44269502 + 1.92596e-8
  const float r = fmaf(x, 1.92596299e-8f, fmaf(x, 1.44269502f, -y));
  const float e = __builtin_amdgcn_exp2f(y);
  return fabsf(y) < 150.0f ? fmaf(e, r * 0.693147181f, e) : e;   // far out: 0, infinity or NaN as it is
}

// softplus(raw + bias) = max(v, 0) + log(1 + t), t = exp(-|v|), with the sum's
// rounding error (Knuth's TwoSum) carried to t.  log(1 + t) = 2 artanh(s), s = t / (2 + t)
// <= 1/3, by its series up to s^15: small dt keep their relative accuracy.
__device__ __forceinline__ float prompt_dt(float raw, float bias, int softplus) {
  const float v = raw + bias;
  if (!softplus) return v;
  const float bb = v - raw;
  // (an infinite v has no rounding error: softplus is 0 or infinity)
  const float lo = fabsf(v) < __builtin_inff() ? (raw - (v - bb)) + (bias - bb) : 0.0f;
  const float t0 = exp_near(-fabsf(v));
  const float t = fmaf(t0, v > 0.0f ? -lo : lo, t0);
  const float d = 2.0f + t;
  float rc = __builtin_amdgcn_rcpf(d);
  rc = fmaf(rc, fmaf(-d, rc, 1.0f), rc);
  const float s = t * rc, q = s * s;
  float p = 2.0f / 15.0f;
  p = fmaf(p, q, 2.0f / 13.0f);
  p = fmaf(p, q, 2.0f / 11.0f);
  p = fmaf(p, q, 2.0f / 9.0f);
  p = fmaf(p, q, 2.0f / 7.0f);
  p = fmaf(p, q, 2.0f / 5.0f);
  p = fmaf(p, q, 2.0f / 3.0f);
  const float l = fmaf(s * q, p, 2.0f * s);
  return v > 0.0f ? v + (lo + l) : l;
}

// v of the lane n places up (n < 0: down) in the lane's row of 16, 0 past its end.
template <int n>
__device__ __forceinline__ float row_shift(float v) {
  constexpr int ctrl = n > 0 ? 0x110 + n : 0x100 - n;   // row_shr : row_shl
  return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), ctrl, 0xf, 0xf, true));
}

// Selections by masks in vector registers: the chunk kernel's scalar registers are all taken, and
// further lane masks there would be spilled inside its loop.
__device__ __forceinline__ int lane_mask(bool on) {
  int m = on ? -1 : 0;
  asm("" : "+v"(m));   // not folded back into a compare
  return m;
}
__device__ __forceinline__ float and_bits(float v, int m) { return __int_as_float(__float_as_int(v) & m); }

template <int IT, int ST, int N, bool kStateOnly>
__global__ __launch_bounds__(kLinBlock, IT == kF32 ? 1 : 2) void linattn_chunk_kernel(LinArgs a) {
  typedef typename Mma<IT>::elem elem;
  typedef typename Mma<IT>::frag frag;
  constexpr int NT = N / 16;
  constexpr int KS = N / 32;
  constexpr int es = sizeof(elem);
  constexpr int ss = sizeof(typename Mma<ST>::elem);
  // parts of w_j x_j in the update: bf16 takes 8 bits a part, enough for an fp32 state or 16 for a
  // state that is stored in 16 bits.  fp16 takes 11, scaled by a power of two that brings the state row's
  // largest term of the chunk below 2^15; weights fall by any factor inside a chunk, so the second part is
  // scaled by another 2^12 and summed apart: 22 bits of terms down to 2^-29 of the largest, and
  // 2^-51 of the largest below (unscaled, a term at 2^-26 kept 13 bits; the sum apart costs 5%)
  constexpr int kParts = IT == kF32 ? 1 : (IT == kBF16 && ST == kF32 ? 3 : 2);
  __shared__ LinLds<IT, N> L;
  const int tid = threadIdx.x, lane = tid & 63, g = lane >> 4, li = lane & 15;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  // Each XCD takes a range of heads of every stretch, so that the heads of a
  // B/C group meet in its L2 and ragged lengths spread evenly; when the heads
  // do not divide among the XCDs, a contiguous range of items.
  const int ptiles = a.dim / kLinP, units = a.H * ptiles;
  int unit, rest;
  if (units % 8 == 0) {
    const int per = units / 8, i = blockIdx.x / 8;
    unit = blockIdx.x % 8 * per + i % per;
    rest = i / per;
  } else {
    const int item = xcd_order(blockIdx.x, gridDim.x);
    unit = item % units;
    rest = item / units;
  }
  const int pt0 = unit % ptiles, h = unit / ptiles;
  const int seg = rest % a.nseg, s = rest / a.nseg;
  const LinSeq q = lin_seq(a, s);
  if (!q.live) return;
  const int t0 = seg * a.seg_len;
  const int t1 = q.len - t0 < a.seg_len ? q.len : t0 + a.seg_len;
  if (kStateOnly ? (q.len - t0 <= a.seg_len) : (seg > 0 && t0 >= q.len)) return;

  const float A = sload(a.A + h);
  const float Dh = a.D != nullptr ? sload(a.D + h) : 0.0f;
  const float bias = a.dt_bias != nullptr ? sload(a.dt_bias + h) : 0.0f;
  const int grp = h / a.hpg;
  const int64_t tile = (static_cast<int64_t>(h) * a.dim + pt0 * kLinP) * N;   // of this workgroup inside a slot
  const int64_t wtile = static_cast<int64_t>(a.H) * a.dim * N;
  // lane's place in the state: row p = 16 wave + li, columns 16 nt + 4g
  const int64_t sat = static_cast<int64_t>(16 * wave + li) * N + 4 * g;
  char* const slot_state = a.state + (q.slot * a.state_stride + tile) * ss;

  f32x4 S[NT];
  if constexpr (kStateOnly) {
#pragma unroll
    for (int n = 0; n < NT; ++n) S[n] = f32x4{0, 0, 0, 0};
  } else if (a.nseg > 1) {
    const float* p = a.ws_state + (static_cast<int64_t>(s) * a.nseg + seg) * wtile + tile + sat;
#pragma unroll
    for (int n = 0; n < NT; ++n) S[n] = *reinterpret_cast<const f32x4*>(p + 16 * n);
  } else if (a.load_state == nullptr || sload(a.load_state + s) != 0) {
#pragma unroll
    for (int n = 0; n < NT; ++n) S[n] = load_state4<ST>(slot_state + (sat + 16 * n) * ss);
  } else {
#pragma unroll
    for (int n = 0; n < NT; ++n) S[n] = f32x4{0, 0, 0, 0};
  }

  Stage<IT, kLinP> xr;
  Stage<IT, N> br;
  frag cr[KS];
  const int64_t hx = static_cast<int64_t>(h) * a.dim + pt0 * kLinP;
  const uint32_t xb = static_cast<uint32_t>(a.x_stride * es), Bb = static_cast<uint32_t>(a.B_stride * es);
  const uint32_t cb = static_cast<uint32_t>(a.C_stride * es), zb = static_cast<uint32_t>(a.z_stride * es);
  const uint32_t yb = static_cast<uint32_t>(a.y_stride * es);
  // addresses of the chunk to load next (x, B, C) and of the current one (z, y)
  const int64_t first = q.start + t0;
  const char* px = a.x + (first * a.x_stride + hx) * es;
  const char* pB = a.B + (first * a.B_stride + static_cast<int64_t>(grp) * N) * es;
  const char* pC = a.C + (first * a.C_stride + static_cast<int64_t>(grp) * N) * es;
  const char* pz = a.z + (first * a.z_stride + hx) * es;
  char* py = a.y + (first * a.y_stride + hx) * es;
  xr.init(xb, tid);
  br.init(Bb, tid);
  const uint32_t c_at = (16 * wave + li) * cb + 8 * g * es, z_at = (16 * wave + li) * zb + 8 * g * es;
  auto fetch = [&](int t) {
    const int rows = t1 - t < kLinQ ? t1 - t : kLinQ;
    xr.load(px, xb, rows);
    br.load(pB, Bb, rows);
    px += static_cast<int64_t>(kLinQ) * xb;
    pB += static_cast<int64_t>(kLinQ) * Bb;
  };
  auto fetch_C = [&](int t) {   // C rows of the wavefront's tokens: column i = 16 wave + li
    const int rows = t1 - t < kLinQ ? t1 - t : kLinQ;
    const rsrc_t rc = make_rsrc(pC, (rows - 1) * cb + N * es);
    pC += static_cast<int64_t>(kLinQ) * cb;
#pragma unroll
    for (int k = 0; k < KS; ++k) {
      const uint32_t at = c_at + 32 * k * es;
      if constexpr (IT == kF32) {
        const u32x4 u = bload16<false>(rc, at, 0), v = bload16<false>(rc, at + 16, 0);
        cr[k] = __builtin_bit_cast(frag, u32x8{u.x, u.y, u.z, u.w, v.x, v.y, v.z, v.w});
      } else {
        cr[k] = __builtin_bit_cast(frag, bload16<false>(rc, at, 0));
      }
    }
  };
  // raw dt of the wavefront's chunk of the four that start at t (lane = token)
  auto fetch_dt = [&](int t) {
    float v = 1.0f;
    const int left = t1 - t - kLinQ * wave;
    if (a.dt != nullptr && left > 0) {
      const int rows = left < kLinQ ? left : kLinQ;
      const uint32_t sb = static_cast<uint32_t>(a.dt_stride) * 4;
      const rsrc_t r = make_rsrc(a.dt + (q.start + t + kLinQ * wave) * a.dt_stride + h, (rows - 1) * sb + 4);
      v = bload_f32(r, lane * sb, 0);
    }
    return v;
  };
  // all bits set where the token one (two) before the lane's is in its group of 4, and where the
  // group of keys 4g .. 4g + 3 is an earlier one than the lane's token's
  const int in_group1 = lane_mask((lane & 3) >= 1), in_group2 = lane_mask((lane & 3) >= 2), earlier = lane_mask(g < li >> 2);
  // Each wavefront turns one chunk's dt into its decays and weights.  Sums of dt A run
  // inside tiles of 16 tokens (lane rows), forwards and backwards, and the tiles' totals
  // multiply as exponentials; inside a tile, the sums between two tokens are put together from
  // groups of 4.  No exponent is a difference of sums: nothing cancels however far a token
  // decays, and an infinite A leaves each token its own term.
  auto scan_dt = [&](int t, float raw) {
    const bool in = t + kLinQ * wave + lane < t1;
    float dtv = a.dt != nullptr ? prompt_dt(raw, bias, a.dt_softplus) : 1.0f;
    dtv = in ? dtv : 0.0f;
    const float da = in ? dtv * A : 0.0f;
    float f = da, r = da;   // inclusive sums up to, and from, the lane's token
    f += row_shift<1>(f);
    r += row_shift<-1>(r);
    f += row_shift<2>(f);
    r += row_shift<-2>(r);
    f += row_shift<4>(f);
    r += row_shift<-4>(r);
    f += row_shift<8>(f);
    r += row_shift<-8>(r);
    float T[4], E[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      T[k] = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(f), 16 * k + 15));
      E[k] = exp_near(T[k]);
    }
    float e = exp_near(f), c = in ? exp_near(row_shift<-1>(r)) * dtv : 0.0f;
    float b = da + and_bits(row_shift<1>(da), in_group1);
    b += and_bits(row_shift<2>(b), in_group2);   // from the start of the lane's group of 4
    const float T4 = __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(b), 0xff, 0xf, 0xf, true));   // whole group
    L.da[wave][lane] = da * 1.44269504f;
    L.since[wave][0][lane] = b * 1.44269504f;
    b += row_shift<4>(T4);
    L.since[wave][1][lane] = b * 1.44269504f;
    b += row_shift<8>(T4);
    L.since[wave][2][lane] = b * 1.44269504f;
    L.lr[wave][lane] = f * 1.44269504f;
    L.dt[wave][lane] = dtv;
#pragma unroll
    for (int k = 0; k < 3; ++k) {
      e *= lane >= 16 * (k + 1) ? E[k] : 1.0f;
      L.before[wave][k][lane] = lane < 16 * (k + 1) ? c : 0.0f;
      c *= lane < 16 * (k + 1) ? E[k + 1] : 1.0f;
    }
    L.e[wave][lane] = e;
    L.w[wave][lane] = c;
    if (lane == 0) {
      L.decay[wave] = (E[0] * E[1]) * (E[2] * E[3]);
      L.total[wave] = (T[0] + T[1]) + (T[2] + T[3]);
    }
  };

  double seg_total = 0.0;
  float dtr = 1.0f;
  if (t0 < t1) {
    dtr = fetch_dt(t0);
    fetch(t0);
    if constexpr (!kStateOnly) fetch_C(t0);
  }
  for (int t = t0; t < t1; t += kLinQ) {
    const int rows = t1 - t < kLinQ ? t1 - t : kLinQ;
    const int c4 = ((t - t0) / kLinQ) & 3;
    if (t > t0) __syncthreads();   // every read of the previous chunk's tiles is done
    xr.store(L.Xs, LinLds<IT, N>::kP, tid);
    br.store(L.Bs, LinLds<IT, N>::kN, tid);
    if constexpr (!kStateOnly) {
      float sc = 1.0f;
      if constexpr (IT == kF16) {   // bring each state row into the range of fp16
        float m = 0.0f;
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int r = 0; r < 4; ++r) m = fmaxf(m, fabsf(S[n][r]));
        const int k = scale_exp(max_groups(m), 12);
        sc = pow2i(k);
        if (g == 0) L.sinv[16 * wave + li] = pow2i(-k);
      }
#pragma unroll
      for (int n = 0; n < NT; ++n)
        narrow4<IT>(L.Ss + (16 * wave + li) * LinLds<IT, N>::kS + 16 * n + 4 * g, IT == kF16 ? S[n] * sc : S[n]);
    }
    if (c4 == 0) scan_dt(t, dtr);
    __syncthreads();
    if (kStateOnly && t + kLinQ < t1) fetch(t + kLinQ);
    if (c4 == 2) dtr = fetch_dt(t + 2 * kLinQ);

    if constexpr (!kStateOnly) {
      const int i = 16 * wave + li;
      const bool has_z = a.z != nullptr;
      u32x4 zw[IT == kF32 ? 4 : 2];
      if (has_z) {
        const rsrc_t rz = make_rsrc(pz, (rows - 1) * zb + kLinP * es);
        pz += static_cast<int64_t>(kLinQ) * zb;
#pragma unroll
        for (int k = 0; k < (IT == kF32 ? 4 : 2); ++k)
          zw[k] = bload16<false>(rz, z_at + (IT == kF32 ? row_of(k, 0) : 32 * k) * es, 0);
      }
      // masked, decay-weighted scores M^T[j][i], j = 16 jt + 4g + r
      f32x4 M[4], Y[4];
      const float lri = L.lr[c4][i];
      const float later = L.since[c4][g < li >> 2 ? (li >> 2) - 1 - g : 0][i];
      const f32x4 a4 = *reinterpret_cast<const f32x4*>(L.da[c4] + 16 * wave + 4 * g);
      const f32x4 dj = *reinterpret_cast<const f32x4*>(L.dt[c4] + 16 * wave + 4 * g);
      // scores (4 tiles of 16 tokens), then the starting state's part (4 tiles of 16 rows): the
      // next tile's fragments are read while the matrix cores take the current ones
      frag f[2][KS];
      auto read = [&](int u, frag (&to)[KS]) {
        const elem* src = u < 4 ? L.Bs + (16 * u + li) * LinLds<IT, N>::kN : L.Ss + row_of(u - 4, li) * LinLds<IT, N>::kS;
#pragma unroll
        for (int k = 0; k < KS; ++k) to[k] = frag_row<IT>(src + 32 * k + 8 * g);
      };
      read(0, f[0]);
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        if (u < 7) read(u + 1, f[(u + 1) & 1]);
        f32x4 acc = f32x4{0, 0, 0, 0};
#pragma unroll
        for (int k = 0; k < KS; ++k) acc = mma<IT>(f[u & 1][k], cr[k], acc);
        if (u < 4) M[u] = acc;
        else Y[u - 4] = acc;
        __builtin_amdgcn_sched_barrier(0);
      }
      if (t + kLinQ < t1) {
        fetch(t + kLinQ);
        fetch_C(t + kLinQ);
      }
      const float ai = __builtin_amdgcn_exp2f(lri);
#pragma unroll
      for (int jt = 0; jt < 4; ++jt) {
        if (jt < wave) {          // earlier tiles: every token is visible
          M[jt] *= *reinterpret_cast<const f32x4*>(L.before[c4][wave - 1] + 16 * jt + 4 * g) * ai;
        } else if (jt == wave) {  // the diagonal
          // log decay from token j to token i > j: the tokens after j in j's group of 4 (j = 4g + r),
          // and those of later groups up to i
          f32x4 d;
          d[3] = and_bits(later, earlier);
#pragma unroll
          for (int r = 2; r >= 0; --r) d[r] = d[r + 1] + (4 * g + r + 1 <= li ? a4[r + 1] : 0.0f);
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const float v = M[jt][r] * (__builtin_amdgcn_exp2f(d[r]) * dj[r]);
            M[jt][r] = 4 * g + r <= li ? v : 0.0f;
          }
        } else {
          M[jt] = f32x4{0, 0, 0, 0};
        }
      }
      int mk = 0;
      if constexpr (IT == kF16) {   // one power of two for the lane's column of M
        float m = 0.0f;
#pragma unroll
        for (int jt = 0; jt < 4; ++jt)
#pragma unroll
          for (int r = 0; r < 4; ++r) m = fmaxf(m, fabsf(M[jt][r]));
        mk = scale_exp(max_groups(m), 12);
        const float ms = pow2i(mk);
#pragma unroll
        for (int jt = 0; jt < 4; ++jt) M[jt] *= ms;
      }
      const float ei = L.e[c4][i], mi = pow2i(-mk);
      f32x4 X[4];
      const frag m0 = to_frag<IT>(stack(M[0], M[1])), m1 = to_frag<IT>(stack(M[2], M[3]));
#pragma unroll
      for (int p = 0; p < 4; ++p) {
        X[p] = mma<IT>(frag_col<IT, 8>(L.Xs, LinLds<IT, N>::kP, 0, row_of(p, 0), lane), m0, f32x4{0, 0, 0, 0});
        X[p] = mma<IT>(frag_col<IT, 8>(L.Xs, LinLds<IT, N>::kP, 32, row_of(p, 0), lane), m1, X[p]);
      }
      const f32x4 xs = (X[0] + X[1]) + (X[2] + X[3]);
      if (__builtin_expect(__ballot(!(fabsf((xs[0] + xs[1]) + (xs[2] + xs[3])) < __builtin_inff())) != 0, 0)) {
        // a non-finite x may have met the zero weight of a later token
#pragma unroll
        for (int p = 0; p < 4; ++p) {
          X[p] = mma_seen<IT>(frag_col<IT, 8>(L.Xs, LinLds<IT, N>::kP, 0, row_of(p, 0), lane), m0, f32x4{0, 0, 0, 0});
          X[p] = mma_seen<IT>(frag_col<IT, 8>(L.Xs, LinLds<IT, N>::kP, 32, row_of(p, 0), lane), m1, X[p]);
        }
      }
      elem* yp = reinterpret_cast<elem*>(py + i * yb) + 8 * g;
      py += static_cast<int64_t>(kLinQ) * yb;
#pragma unroll
      for (int p = 0; p < 4; ++p) {
        if constexpr (IT == kF16) Y[p] *= *reinterpret_cast<const f32x4*>(L.sinv + row_of(p, 4 * g));
        Y[p] = Y[p] * ei + X[p] * mi;
      }
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const f32x8 xi = from_frag<IT>(frag_row<IT>(L.Xs + i * LinLds<IT, N>::kP + 32 * k + 8 * g));
        f32x8 v = stack(Y[2 * k], Y[2 * k + 1]) + xi * Dh;
        if (has_z) {
          f32x8 zi;
          if constexpr (IT == kF32) zi = __builtin_bit_cast(f32x8, u32x8{zw[2 * k].x, zw[2 * k].y, zw[2 * k].z, zw[2 * k].w, zw[2 * k + 1].x, zw[2 * k + 1].y, zw[2 * k + 1].z, zw[2 * k + 1].w});
          else zi = from_frag<IT>(__builtin_bit_cast(frag, zw[k]));
#pragma unroll
          for (int e = 0; e < 8; ++e) v[e] *= silu(zi[e]);
        }
        if (i < rows) {
          if constexpr (IT == kF32) {
            *reinterpret_cast<f32x4*>(yp + 32 * k) = f32x4{v[0], v[1], v[2], v[3]};
            *reinterpret_cast<f32x4*>(yp + 32 * k + 4) = f32x4{v[4], v[5], v[6], v[7]};
          } else {
            *reinterpret_cast<u32x4*>(yp + 32 * k) = __builtin_bit_cast(u32x4, to_frag<IT>(v));
          }
        }
      }
    }

    // state: S^T[n][p] of the wavefront's 16 rows p = 16 wave + li
    const float decay = L.decay[c4];
    if constexpr (kStateOnly) seg_total += L.total[c4];
    frag u0[2], u1[2], u2[2];
    f32x8 wx[2];
    int sk = 0;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const f32x4 w0 = *reinterpret_cast<const f32x4*>(L.w[c4] + 32 * k + 4 * g);
      const f32x4 w1 = *reinterpret_cast<const f32x4*>(L.w[c4] + 32 * k + 16 + 4 * g);
      wx[k] = from_frag<IT>(frag_col<IT>(L.Xs, LinLds<IT, N>::kP, 32 * k, 16 * wave, lane)) * stack(w0, w1);
    }
    if constexpr (IT == kF16) {
      float m = 0.0f;
#pragma unroll
      for (int k = 0; k < 2; ++k)
#pragma unroll
        for (int e = 0; e < 8; ++e) m = fmaxf(m, fabsf(wx[k][e]));
      sk = scale_exp(max_groups(m), 14);
    }
    const float up = pow2i(sk), down = pow2i(-sk);
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const f32x8 v = IT == kF16 ? wx[k] * up : wx[k];
      if constexpr (IT == kBF16) {
        f32x8 left = v;
        u0[k] = take_bf16(left);
        u1[k] = take_bf16(left);
        if constexpr (kParts > 2) u2[k] = take_bf16(left);
      } else {
        u0[k] = to_frag<IT>(v);
        if constexpr (kParts > 1) u1[k] = to_frag<IT>((v - from_frag<IT>(u0[k])) * 0x1p12f);
      }
    }
    const float dup = IT == kF16 ? decay * up : decay;
#pragma unroll
    for (int n = 0; n < NT; ++n) S[n] *= dup;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      f32x4 low = f32x4{0, 0, 0, 0};   // fp16: the second parts' sum
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const frag b = frag_col<IT>(L.Bs, LinLds<IT, N>::kN, 32 * k, 16 * n, lane);
        if constexpr (kParts > 2) S[n] = mma<IT>(b, u2[k], S[n]);
        if constexpr (IT == kF16) low = mma<IT>(b, u1[k], low);
        else if constexpr (kParts > 1) S[n] = mma<IT>(b, u1[k], S[n]);
        S[n] = mma<IT>(b, u0[k], S[n]);
      }
      if constexpr (IT == kF16) S[n] = (S[n] + low * 0x1p-12f) * down;
    }
  }

  if constexpr (kStateOnly) {
    float* p = a.ws_state + (static_cast<int64_t>(s) * a.nseg + seg + 1) * wtile + tile + sat;
#pragma unroll
    for (int n = 0; n < NT; ++n) *reinterpret_cast<f32x4*>(p + 16 * n) = S[n];
    if (tid == 0 && pt0 == 0)
      a.ws_decay[(static_cast<int64_t>(s) * a.nseg + seg) * a.H + h] = static_cast<float>(seg_total);
  } else if (t1 == q.len) {
#pragma unroll
    for (int n = 0; n < NT; ++n) store_state4<ST>(slot_state + (sat + 16 * n) * ss, S[n]);
  }
}

// Scan over stretches: workspace entry k becomes the state at the start of stretch k
// (entry k + 1 held stretch k's own state from zero).  One thread a quartet of
// state elements of one (sequence, head).
template <int ST>
__global__ __launch_bounds__(kLinBlock) void linattn_scan_kernel(LinArgs a, int elems) {
  constexpr int ss = sizeof(typename Mma<ST>::elem);
  const int h = blockIdx.y, s = blockIdx.z;
  const LinSeq q = lin_seq(a, s);
  if (!q.live) return;
  const int at = (blockIdx.x * kLinBlock + threadIdx.x) * 4;
  if (at >= elems) return;
  const int64_t hs = static_cast<int64_t>(h) * elems + at, wtile = static_cast<int64_t>(a.H) * elems;
  f32x4 run = f32x4{0, 0, 0, 0};
  if (a.load_state == nullptr || sload(a.load_state + s) != 0)
    run = load_state4<ST>(a.state + (q.slot * a.state_stride + hs) * ss);
  float* w = a.ws_state + static_cast<int64_t>(s) * a.nseg * wtile + hs;
  *reinterpret_cast<f32x4*>(w) = run;
  const float* dec = a.ws_decay + static_cast<int64_t>(s) * a.nseg * a.H + h;
  const int steps = q.len > 0 ? (q.len - 1) / a.seg_len : 0;   // stretches that another one follows
  constexpr int U = 8;   // loads in flight
  for (int k0 = 0; k0 < steps; k0 += U) {
    f32x4 own[U];
    float d[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int k = k0 + u < steps ? k0 + u : steps - 1;
      own[u] = *reinterpret_cast<const f32x4*>(w + (k + 1) * wtile);
      d[u] = sload(dec + static_cast<int64_t>(k) * a.H);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (k0 + u < steps) {
        run = run * exp_near(d[u]) + own[u];
        *reinterpret_cast<f32x4*>(w + (k0 + u + 1) * wtile) = run;
      }
    }
  }
}

// Single-token form: one workgroup a (request, head, 64 state rows), 16 rows a
// wavefront.  The state streams through registers once (16-byte non-temporal loads and
// stores, all of a wavefront's rows in flight); each lane folds its columns
// and the row's readout is summed over the lanes that share it.  Bound by memory:
// 256 requests of 256 heads of 64 x 128 bf16 in 0.369 ms, 5.9 TB/s read and written; one
// request 4.2 us, most of it the launch.
template <int IT, int ST, int N>
__global__ __launch_bounds__(kLinBlock) void linattn_step_kernel(LinArgs a) {
  typedef typename Mma<IT>::elem elem;
  constexpr int ss = sizeof(typename Mma<ST>::elem);
  constexpr int EV = 16 / ss;            // columns a lane
  constexpr int LPR = N / EV;            // lanes a row
  constexpr int RPP = 64 / LPR;          // rows a pass
  constexpr int PASSES = 16 / RPP;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int ptiles = a.dim / kLinP;
  const int pt0 = blockIdx.x % ptiles, h = (blockIdx.x / ptiles) % a.H, b = blockIdx.x / (ptiles * a.H);
  const int slot = sload(a.slots + b);
  if (slot == a.pad || slot < 0 || slot >= a.num_slots) return;
  const int row0 = pt0 * kLinP + 16 * wave, cc = lane % LPR, rr = lane / LPR;
  char* const st0 = a.state + (slot * a.state_stride + (static_cast<int64_t>(h) * a.dim + row0 + rr) * N + cc * EV) * ss;
  u32x4 raw[PASSES];
#pragma unroll
  for (int p = 0; p < PASSES; ++p) raw[p] = ld<true, u32x4>(st0 + p * (RPP * N * ss));
  const int grp = h / a.hpg;
  const elem* Bp = reinterpret_cast<const elem*>(a.B) + b * a.B_stride + static_cast<int64_t>(grp) * N + cc * EV;
  const elem* Cp = reinterpret_cast<const elem*>(a.C) + b * a.C_stride + static_cast<int64_t>(grp) * N + cc * EV;
  f32x4 Bv[EV / 4], Cv[EV / 4];
#pragma unroll
  for (int k = 0; k < EV / 4; ++k) {
    Bv[k] = widen4<IT>(Bp + 4 * k);
    Cv[k] = widen4<IT>(Cp + 4 * k);
  }
  float dt = 1.0f;
  if (a.dt != nullptr)
    dt = prompt_dt(sload(a.dt + b * a.dt_stride + h), a.dt_bias != nullptr ? sload(a.dt_bias + h) : 0.0f, a.dt_softplus);
  const float decay = expf(dt * sload(a.A + h));
  const float Dh = a.D != nullptr ? sload(a.D + h) : 0.0f;
  const int64_t hx = static_cast<int64_t>(h) * a.dim + row0 + rr;
  const elem* xp = reinterpret_cast<const elem*>(a.x) + b * a.x_stride + hx;
  const elem* zp = a.z != nullptr ? reinterpret_cast<const elem*>(a.z) + b * a.z_stride + hx : nullptr;
  elem* yp = reinterpret_cast<elem*>(a.y) + b * a.y_stride + hx;
  float xv[PASSES], zv[PASSES];
#pragma unroll
  for (int p = 0; p < PASSES; ++p) {
    xv[p] = elem_to_float<IT>(xp[p * RPP]);
    zv[p] = zp != nullptr ? elem_to_float<IT>(zp[p * RPP]) : 0.0f;
  }
#pragma unroll
  for (int p = 0; p < PASSES; ++p) {
    const float dx = dt * xv[p];
    float sum = 0.0f;
    u32x4 o;
    if constexpr (ST == kF32) {
      const f32x4 v = __builtin_bit_cast(f32x4, raw[p]) * decay + Bv[0] * dx;
#pragma unroll
      for (int e = 0; e < 4; ++e) sum = fmaf(v[e], Cv[0][e], sum);
      o = __builtin_bit_cast(u32x4, v);
    } else {
      const f32x8 old = from_frag<ST>(__builtin_bit_cast(typename Mma<ST>::frag, raw[p]));
      const f32x8 v = old * decay + stack(Bv[0], Bv[EV / 4 - 1]) * dx;
#pragma unroll
      for (int e = 0; e < 4; ++e) sum = fmaf(v[e], Cv[0][e], sum);
#pragma unroll
      for (int e = 0; e < 4; ++e) sum = fmaf(v[4 + e], Cv[EV / 4 - 1][e], sum);
      o = __builtin_bit_cast(u32x4, to_frag<ST>(v));
    }
    st<true>(st0 + p * (RPP * N * ss), o);
#pragma unroll
    for (int d = 1; d < LPR; d <<= 1) sum += __shfl_xor(sum, d);
    if (cc == 0) {
      float v = fmaf(Dh, xv[p], sum);
      if (zp != nullptr) v *= silu(zv[p]);
      if constexpr (IT == kF32) yp[p * RPP] = v;
      else if constexpr (IT == kBF16) yp[p * RPP] = __builtin_bit_cast(uint16_t, static_cast<__bf16>(v));
      else yp[p * RPP] = __builtin_bit_cast(uint16_t, static_cast<_Float16>(v));
    }
  }
}

}  // namespace rssm
