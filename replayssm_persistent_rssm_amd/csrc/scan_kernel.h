// scan_kernel.h -- gfx950 kernels of the selective state-space scan: ragged
// prompts and single tokens.
//
// The decay of each (token, channel, state) is an exponential of its own, so no matrix product does this
// work: one exponential, two products and two multiply-adds for each of them on the vector ALUs are the
// bound, and everything else is arranged so as not to add to it.
//
// scan_kernel: a wavefront owns 16 channels of a sequence and all their states in registers: lane 16 g + j
// has states 16 m + 4 g .. 16 m + 4 g + 3 of channel j.  It walks the tokens in tiles of 16.
//  * Inputs of a tile come as lane 16 g + j = token j, channels 4g .. 4g + 3 (x, dt, z): one load an input, each step
//    size computed once.  Rows past the end read as zeros by the size of their buffer.
//  * Step sizes go to the channels' lanes through LDS (16 x 16 floats of the wavefront's own, no barrier).
//  * d x B is an outer product of 16 channels and 16 states a token: a matrix instruction gives four tokens of it (four
//    blocks of 16 x 16 with one product each, exact to one rounding), in the layout that the states are in.
//  * C_t is the same for all 16 channels: it is broadcast from lane t of each row of 16 by the instruction that
//    multiplies it (row broadcast), at no cost.
//  * The sums over the four groups of lanes are taken for four tokens at once by swapping halves and rows of lanes
//    (6 instructions for 4 tokens), and go back to the tile's layout through LDS for skip, gate and store.
// When sequences and channels leave compute units empty, the token axis is split: scan_kernel<FOLD> gives
// each stretch's own end state and the sum of its step sizes (a decay over the stretch is exp(A sum)), and
// the main kernel starts each stretch from those of the stretches before it.  The state pool is read by one launch
// and written by the other.
// 12 ragged prompts up to 2,011 tokens, 8,192 bf16 channels of 16 states: 417 us, the vector ALUs busy throughout (416
// instructions a tile, 256 of them the four an element); one of 16,384 tokens, 4,096 channels: 413 us in 24
// stretches, 169 us in the fold and 243 in the main kernel (many calls in turn; 470 in the first few after a pause, at
// lower clocks).
// scan_step_kernel: a lane has 16 bytes of a channel's states; bound by reading and writing the state.
#pragma once

#include "mma_device.h"

namespace rssm {

struct ScanArgs {
  char* state;
  const float* A;
  const float* D;             // or null
  const float* dt_bias;       // or null
  const char* x;
  const char* dt;
  const char* B;
  const char* C;
  const char* z;              // or null
  char* y;
  const int32_t* slots;
  const int32_t* seq_start;
  const int32_t* load_state;  // or null
  float* ws_h;                // [num_seqs][nseg][channels][N] (nseg > 1): ends of stretches; of the last one the start of the first
  float* ws_d;                // [num_seqs][nseg][channels]
  int64_t state_stride, x_stride, dt_stride, B_stride, C_stride, z_stride, y_stride;   // elements
  int32_t num_seqs, num_tokens, channels, groups, per_group, num_slots, pad, max_seq_len, dt_softplus, state_dtype;
  int32_t nseg, seg_len;      // stretches of the token axis and their length (a multiple of 16)
  int32_t blocks;             // channel blocks
};

constexpr int kScanBlock = 256;
constexpr int kScanChannels = 64;    // a workgroup of scan_kernel, 16 a wavefront
constexpr int kScanShortChannels = 16;   // a workgroup of scan_short_kernel, 4 a wavefront
constexpr int kScanTile = 16;        // tokens
constexpr int kScanPitch = 20;       // floats between rows of an LDS tile: 16-byte pieces of 16 rows on different banks
constexpr float kLog2e = 1.44269504088896341f;

// n elements in storage.
template <int IT, int n>
struct ScanRaw {
  static constexpr int kWords = n * static_cast<int>(sizeof(typename Mma<IT>::elem)) / 4;
  uint32_t w[kWords];
  __device__ __forceinline__ void load(const char* p) {
    if constexpr (kWords == 2) {
      const u32x2 v = ld<false, u32x2>(p);
      w[0] = v.x, w[1] = v.y;
    } else {
#pragma unroll
      for (int k = 0; k < kWords; k += 4) {
        const u32x4 v = ld<false, u32x4>(p + k * 4);
        w[k] = v.x, w[k + 1] = v.y, w[k + 2] = v.z, w[k + 3] = v.w;
      }
    }
  }
  __device__ __forceinline__ float get(int i) const {
    if constexpr (IT == kF32) return __uint_as_float(w[i]);
    else if constexpr (IT == kBF16) return __uint_as_float(i & 1 ? w[i / 2] & 0xffff0000u : w[i / 2] << 16);
    else return f16_bits_to_float(i & 1 ? w[i / 2] >> 16 : w[i / 2] & 0xffffu);
  }
};

// Order of the wavefront's own LDS accesses.
__device__ __forceinline__ void scan_wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

// p plus (kFirst: instead of p) the sum of four products C_i h_i with C broadcast from lane T of each row.  The compiler
// broadcasts into products but not into multiply-adds (a move more for each), so these are written out; the first
// instruction covers the wait that a broadcast needs after a vector instruction wrote its source.
template <int T, bool kFirst>
__device__ __forceinline__ float scan_dot4(float p, const float* C, const float* h) {
#define RSSM_ROW " row_newbcast:%c[t] row_mask:0xf bank_mask:0xf\n\t"
  if constexpr (kFirst) {
    asm("s_nop 1\n\t"
        "v_mul_f32_dpp %[p], %[c0], %[h0]" RSSM_ROW
        "v_fmac_f32_dpp %[p], %[c1], %[h1]" RSSM_ROW
        "v_fmac_f32_dpp %[p], %[c2], %[h2]" RSSM_ROW
        "v_fmac_f32_dpp %[p], %[c3], %[h3]" RSSM_ROW
        : [p] "=&v"(p)
        : [c0] "v"(C[0]), [c1] "v"(C[1]), [c2] "v"(C[2]), [c3] "v"(C[3]), [h0] "v"(h[0]), [h1] "v"(h[1]), [h2] "v"(h[2]),
          [h3] "v"(h[3]), [t] "i"(T));
  } else {
    asm("s_nop 1\n\t"
        "v_fmac_f32_dpp %[p], %[c0], %[h0]" RSSM_ROW
        "v_fmac_f32_dpp %[p], %[c1], %[h1]" RSSM_ROW
        "v_fmac_f32_dpp %[p], %[c2], %[h2]" RSSM_ROW
        "v_fmac_f32_dpp %[p], %[c3], %[h3]" RSSM_ROW
        : [p] "+&v"(p)
        : [c0] "v"(C[0]), [c1] "v"(C[1]), [c2] "v"(C[2]), [c3] "v"(C[3]), [h0] "v"(h[0]), [h1] "v"(h[1]), [h2] "v"(h[2]),
          [h3] "v"(h[3]), [t] "i"(T));
  }
#undef RSSM_ROW
  return p;
}

// Lanes 0-31: a summed over lane and lane + 32; lanes 32-63: b likewise.
__device__ __forceinline__ float halves_sum(float a, float b) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(a), __float_as_uint(b), false, false);
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}

// Rows 0 and 2 of 16 lanes: a summed over the row and the next one; rows 1 and 3: b likewise.
__device__ __forceinline__ float rows_sum(float a, float b) {
  const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(a), __float_as_uint(b), false, false);
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}

// One element of the state pool, by its dtype.
__device__ __forceinline__ float scan_state_load(const char* base, int64_t at, int dtype) {
  if (dtype == kF32) return gload(reinterpret_cast<const float*>(base) + at);
  const uint16_t v = gload(reinterpret_cast<const uint16_t*>(base) + at);
  return dtype == kBF16 ? elem_to_float<kBF16>(v) : elem_to_float<kF16>(v);
}

__device__ __forceinline__ void scan_state_store(char* base, int64_t at, int dtype, float v) {
  if (dtype == kF32) {
    gstore(reinterpret_cast<float*>(base) + at, v);
  } else {
    const uint16_t h = dtype == kBF16 ? __builtin_bit_cast(uint16_t, static_cast<__bf16>(v))
                                      : __builtin_bit_cast(uint16_t, static_cast<_Float16>(v));
    gstore(reinterpret_cast<uint16_t*>(base) + at, h);
  }
}

// A log2(e), with -infinity as the most negative number: a step of size 0 then decays by exp2(-0) = 1.  (A NaN stays.)
__device__ __forceinline__ float scan_rate(float A) {
  const float v = A * kLog2e;
  return v < -3.40282347e38f ? -3.40282347e38f : v;
}

// softplus(v) = max(v, 0) + log(1 + t), t = exp(-|v|); log(1 + t) / t on [0, 1] is the polynomial through its values
// at the ten Chebyshev points (off by 1.4e-8 of itself, 1.3e-7 with its roundings): small steps keep
// their relative accuracy.
__device__ __forceinline__ float scan_step_size(float raw, float bias, int softplus) {
  const float v = raw + bias;
  if (!softplus) return v;
  const float t = __builtin_amdgcn_exp2f(-fabsf(v) * kLog2e);
  float p = -0.0031760570127516985f;
  p = fmaf(p, t, 0.019542526453733444f);
  p = fmaf(p, t, -0.056373611092567444f);
  p = fmaf(p, t, 0.10543623566627502f);
  p = fmaf(p, t, -0.1526966691017151f);
  p = fmaf(p, t, 0.1966327428817749f);
  p = fmaf(p, t, -0.24951615929603577f);
  p = fmaf(p, t, 0.33329710364341736f);
  p = fmaf(p, t, -0.49999892711639404f);
  p = fmaf(p, t, 1.0f);
  return fmaf(p, t, fmaxf(v, 0.0f));
}

// A tensor's rows of one sequence, a tile of 16 at a time: a buffer that ends with the last row, so that loads past it
// give 0 and stores past it are dropped.  Addresses advance in scalar registers.
struct ScanRows {
  const char* at;          // first row of the tile
  uint32_t step, width;    // bytes between rows (at most 2^26) and in one
  __device__ __forceinline__ void start(const char* base, int64_t row, int64_t stride, int width_bytes, int es) {
    at = base + row * stride * es;
    step = static_cast<uint32_t>(stride * es);
    width = static_cast<uint32_t>(width_bytes);
  }
  __device__ __forceinline__ rsrc_t tile(int rows) const {
    return make_rsrc(at, (static_cast<uint32_t>(rows < kScanTile ? rows : kScanTile) - 1) * step + width);
  }
  __device__ __forceinline__ void next() { at += static_cast<int64_t>(kScanTile) * step; }
};

// 4 elements in storage, at a byte offset of a buffer.
template <int IT>
struct ScanFour {
  static constexpr int kWords = static_cast<int>(sizeof(typename Mma<IT>::elem));
  uint32_t w[kWords];
  __device__ __forceinline__ void load(rsrc_t r, uint32_t off) {
    if constexpr (IT == kF32) {
      const u32x4 v = bload16<false>(r, off, 0);
      w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
    } else {
      const u32x2 v = __builtin_bit_cast(u32x2, __builtin_amdgcn_raw_buffer_load_b64(r, off, 0, 0));
      w[0] = v.x, w[1] = v.y;
    }
  }
  __device__ __forceinline__ float get(int i) const {
    if constexpr (IT == kF32) return __uint_as_float(w[i]);
    else if constexpr (IT == kBF16) return __uint_as_float(i & 1 ? w[i / 2] & 0xffff0000u : w[i / 2] << 16);
    else return f16_bits_to_float(i & 1 ? w[i / 2] >> 16 : w[i / 2] & 0xffffu);
  }
};

template <int IT>
__device__ __forceinline__ uint32_t scan_one_load(rsrc_t r, uint32_t off) {
  if constexpr (IT == kF32) return __builtin_amdgcn_raw_buffer_load_b32(r, off, 0, 0);
  else return __builtin_amdgcn_raw_buffer_load_b16(r, off, 0, 0);
}
template <int IT>
__device__ __forceinline__ float scan_one(uint32_t w) {
  if constexpr (IT == kF32) return __uint_as_float(w);
  else return elem_to_float<IT>(static_cast<uint16_t>(w));
}

typedef float f32x16 __attribute__((ext_vector_type(16)));

constexpr uint32_t kScanNowhere = 0xfffffff0u;   // offset past every buffer

// Sequence with the rank-th longest row range (ties: lower index first), for at most 64 sequences: the long ones start
// first, so that they do not run alone at the end.
__device__ __forceinline__ int scan_by_length(const ScanArgs& a, int rank, int lane) {
  int len = -1;
  if (lane < a.num_seqs) len = gload(a.seq_start + lane + 1) - gload(a.seq_start + lane);
  int before = 0;
  for (int i = 0; i < a.num_seqs; ++i) {
    const int other = __builtin_amdgcn_readlane(len, i);
    before += other > len || (other == len && i < lane) ? 1 : 0;
  }
  return __builtin_ctzll(__ballot(lane < a.num_seqs && before == rank));
}

template <int M>
struct ScanState {
  float A[4 * M], h[4 * M];
};

// Token T of a tile: the states move on; the lane's part of y_t.
template <int M, bool FOLD, int T>
__device__ __forceinline__ float scan_token(const float (&dt)[kScanTile], const float (&C)[4 * M], const f32x16 (&u)[M],
                                            ScanState<M>& s) {
  float p = 0.0f;
#pragma unroll
  for (int m = 0; m < M; ++m) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float e = __builtin_amdgcn_exp2f(dt[T] * s.A[4 * m + i]);
      s.h[4 * m + i] = fmaf(e, s.h[4 * m + i], u[m][4 * (T & 3) + i]);
    }
    if constexpr (!FOLD) p = m == 0 ? scan_dot4<T, true>(p, C, s.h) : scan_dot4<T, false>(p, C + 4 * m, s.h + 4 * m);
  }
  return p;
}

// Tokens 4 Q .. 4 Q + 3.  B: of token 4 Q + g, states 16 m + j; dx: of token 4 Q + g, channel j.
template <int M, bool FOLD, int Q>
__device__ __forceinline__ float scan_four(const float (&dt)[kScanTile], const float (&B)[4][M], const float (&dx)[4],
                                           const float (&C)[4 * M], ScanState<M>& s) {
  f32x16 u[M];
#pragma unroll
  for (int m = 0; m < M; ++m) {
    const f32x16 zero = {0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0};
    u[m] = __builtin_amdgcn_mfma_f32_16x16x1f32(B[Q][m], dx[Q], zero, 0, 0, 0);
  }
  const float p0 = scan_token<M, FOLD, 4 * Q>(dt, C, u, s);
  const float p1 = scan_token<M, FOLD, 4 * Q + 1>(dt, C, u, s);
  const float p2 = scan_token<M, FOLD, 4 * Q + 2>(dt, C, u, s);
  const float p3 = scan_token<M, FOLD, 4 * Q + 3>(dt, C, u, s);
  if constexpr (FOLD) return 0.0f;
  return rows_sum(halves_sum(p0, p2), halves_sum(p1, p3));   // row g: token 4 Q + g
}

// Two wavefronts a SIMD keep the results of the matrix instructions out of the accumulation registers; the widest instance, which
// comes within a few registers of spilling at that, may take one.
template <int IT, int N, bool FOLD>
__global__ __launch_bounds__(kScanBlock, IT == kF32 && N == 64 ? 1 : 2) void scan_kernel(ScanArgs a) {
  constexpr int es = sizeof(typename Mma<IT>::elem);
  constexpr int M = N / 16;
  __shared__ alignas(16) float lds[kScanBlock / 64][3][kScanTile * kScanPitch];
  const int tid = threadIdx.x, lane = tid & 63, j = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  int b = blockIdx.x;
  const int c0 = (b % a.blocks) * kScanChannels + wave * 16;
  b /= a.blocks;
  const int seg = b % a.nseg;
  int s = b / a.nseg;
  if (c0 >= a.channels) return;
  if (a.num_seqs > 1 && a.num_seqs <= 64) s = scan_by_length(a, s, lane);
  const int slot = sload(a.slots + s);
  if (slot == a.pad || slot < 0 || slot >= a.num_slots) return;
  int start = sload(a.seq_start + s), end = sload(a.seq_start + s + 1);
  start = start < 0 ? 0 : (start > a.num_tokens ? a.num_tokens : start);
  end = end < start ? start : (end > a.num_tokens ? a.num_tokens : end);
  const int len = end - start < a.max_seq_len ? end - start : a.max_seq_len;
  const int last = len > 0 ? (len - 1) / a.seg_len : 0;       // the stretch that holds the last token
  if (seg > last || (FOLD && seg == last)) return;
  const int beg = seg * a.seg_len, n = len - beg < a.seg_len ? len - beg : a.seg_len;
  const int64_t tok = start + static_cast<int64_t>(beg);

  const int cj = c0 + j, cg = c0 + 4 * g;                     // the lane's channel, its first channel of a tile's inputs
  const bool has_j = cj < a.channels, has_g = cg < a.channels;
  const int64_t st0 = slot * a.state_stride + static_cast<int64_t>(cj) * N + 4 * g;
  ScanState<M> st;
#pragma unroll
  for (int i = 0; i < 4 * M; ++i) {
    const int n0 = 16 * (i / 4) + i % 4;                      // state of the lane's group
    st.A[i] = has_j ? scan_rate(gload(a.A + static_cast<int64_t>(cj) * N + 4 * g + n0)) : 0.0f;
    st.h[i] = 0.0f;
  }
  // The pool is written by the last stretch, and nothing orders the workgroups of a launch: where there are several
  // stretches the fold of the first one alone reads it, and leaves the state in the last one's workspace entry, which no fold
  // fills.
  const int64_t held = (static_cast<int64_t>(s) * a.nseg + last) * a.channels + cj;
  if (has_j && (FOLD ? seg == 0 : last == 0) && (a.load_state == nullptr || sload(a.load_state + s) != 0)) {
#pragma unroll
    for (int i = 0; i < 4 * M; ++i) st.h[i] = scan_state_load(a.state, st0 + 16 * (i / 4) + i % 4, a.state_dtype);
  }
  if constexpr (FOLD) {
    if (seg == 0) {
#pragma unroll
      for (int i = 0; i < 4 * M; ++i) {
        if (has_j) gstore(a.ws_h + held * N + 4 * g + 16 * (i / 4) + i % 4, st.h[i]);
        st.h[i] = 0.0f;
      }
    }
  } else if (has_j && last > 0) {
#pragma unroll
    for (int i = 0; i < 4 * M; ++i) st.h[i] = gload(a.ws_h + held * N + 4 * g + 16 * (i / 4) + i % 4);
#pragma unroll 4
    for (int k = 0; k < seg; ++k) {
      const int64_t at = (static_cast<int64_t>(s) * a.nseg + k) * a.channels + cj;
      const float sum = gload(a.ws_d + at);
#pragma unroll
      for (int i = 0; i < 4 * M; ++i) {
        // from zero a stretch ends where its fold does, also where its steps together would grow a state past fp32
        const float own = gload(a.ws_h + at * N + 4 * g + 16 * (i / 4) + i % 4);
        st.h[i] = st.h[i] == 0.0f ? own : fmaf(__builtin_amdgcn_exp2f(sum * st.A[i]), st.h[i], own);
      }
    }
  }
  float bias[4], D[4], dsum[4] = {0, 0, 0, 0};
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    bias[r] = a.dt_bias != nullptr && has_g ? gload(a.dt_bias + cg + r) : 0.0f;
    D[r] = a.D != nullptr && has_g ? gload(a.D + cg + r) : 0.0f;
  }
  const int gN = a.groups * N;
  ScanRows xr, dr, zr, Br, Cr, yr;
  xr.start(a.x, tok, a.x_stride, a.channels * es, es);
  dr.start(a.dt, tok, a.dt_stride, a.channels * es, es);
  Br.start(a.B, tok, a.B_stride, gN * es, es);
  const bool gated = a.z != nullptr;
  if constexpr (!FOLD) {
    Cr.start(a.C, tok, a.C_stride, gN * es, es);
    yr.start(a.y, tok, a.y_stride, a.channels * es, es);
    zr.start(gated ? a.z : a.x, tok, gated ? a.z_stride : a.x_stride, a.channels * es, es);
  }
  const uint32_t row = static_cast<uint32_t>(c0 / a.per_group) * N;
  const uint32_t xo = has_g ? j * xr.step + cg * es : kScanNowhere, dto = has_g ? j * dr.step + cg * es : kScanNowhere;
  const uint32_t Bo = g * Br.step + (row + j) * es;
  uint32_t zo = 0, yo = 0, Co = 0;
  if constexpr (!FOLD) {
    zo = has_g ? j * zr.step + cg * es : kScanNowhere;
    yo = has_g ? j * yr.step + cg * es : kScanNowhere;
    Co = j * Cr.step + (row + 4 * g) * es;
  }
  ScanFour<IT> rx, rd, rz, rC[M];
  uint32_t rB[4][M];
  const auto fetch = [&](int rows) {
    rx.load(xr.tile(rows), xo);
    rd.load(dr.tile(rows), dto);
    const rsrc_t rb = Br.tile(rows);
#pragma unroll
    for (int q = 0; q < 4; ++q) {
#pragma unroll
      for (int m = 0; m < M; ++m) rB[q][m] = scan_one_load<IT>(rb, Bo + 4 * q * Br.step + 16 * m * es);
    }
    xr.next();
    dr.next();
    Br.next();
    if constexpr (!FOLD) {
      const rsrc_t rc = Cr.tile(rows);
#pragma unroll
      for (int m = 0; m < M; ++m) rC[m].load(rc, Co + 16 * m * es);
      rz.load(zr.tile(rows), zo);
      Cr.next();
      zr.next();
    }
  };
  if (n > 0) fetch(n);
  float* const sd = lds[wave][0];
  float* const sx = lds[wave][1];
  float* const sy = lds[wave][2];
  for (int t0 = 0; t0 < n; t0 += kScanTile) {
    const bool on = t0 + j < n;
    float x[4], z[4], B[4][M], C[4 * M];
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      x[r] = rx.get(r);
      z[r] = FOLD ? 0.0f : rz.get(r);
      float d = scan_step_size(rd.get(r), bias[r], a.dt_softplus);
      d = on ? d : 0.0f;
      if constexpr (FOLD) dsum[r] += d;
      sd[(4 * g + r) * kScanPitch + j] = d;
      sx[(4 * g + r) * kScanPitch + j] = d * x[r];
    }
#pragma unroll
    for (int q = 0; q < 4; ++q) {
#pragma unroll
      for (int m = 0; m < M; ++m) B[q][m] = scan_one<IT>(rB[q][m]);
    }
#pragma unroll
    for (int i = 0; i < 4 * M; ++i) C[i] = FOLD ? 0.0f : rC[i / 4].get(i % 4);
    if (t0 + kScanTile < n) fetch(n - t0 - kScanTile);
    scan_wave_sync();
    float dt[kScanTile], dx[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const f32x4 d = *reinterpret_cast<const f32x4*>(sd + j * kScanPitch + 4 * q);
#pragma unroll
      for (int e = 0; e < 4; ++e) dt[4 * q + e] = d[e];
      dx[q] = sx[j * kScanPitch + 4 * q + g];
    }
    const float y0 = scan_four<M, FOLD, 0>(dt, B, dx, C, st);
    const float y1 = scan_four<M, FOLD, 1>(dt, B, dx, C, st);
    const float y2 = scan_four<M, FOLD, 2>(dt, B, dx, C, st);
    const float y3 = scan_four<M, FOLD, 3>(dt, B, dx, C, st);
    if constexpr (!FOLD) {
      sy[g * kScanPitch + j] = y0;
      sy[(4 + g) * kScanPitch + j] = y1;
      sy[(8 + g) * kScanPitch + j] = y2;
      sy[(12 + g) * kScanPitch + j] = y3;
      scan_wave_sync();
      f32x4 y = *reinterpret_cast<const f32x4*>(sy + j * kScanPitch + 4 * g);
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        y[r] = fmaf(D[r], x[r], y[r]);
        if (gated) y[r] *= silu(z[r]);
      }
      const rsrc_t ry = yr.tile(n - t0);
      if constexpr (IT == kF32) {
        bstore16<false>(ry, yo, 0, __builtin_bit_cast(u32x4, y));
      } else {
        typename Mma<IT>::elem out[4];
        narrow4<IT>(out, y);
        typedef decltype(__builtin_amdgcn_raw_buffer_load_b64(ry, 0u, 0u, 0)) two;
        two v;
        __builtin_memcpy(&v, out, 8);
        __builtin_amdgcn_raw_buffer_store_b64(v, ry, yo, 0, 0);
      }
      yr.next();
    }
    scan_wave_sync();
  }
  if constexpr (FOLD) {
    const int64_t at = (static_cast<int64_t>(s) * a.nseg + seg) * a.channels;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      float v = dsum[r];
#pragma unroll
      for (int m = 1; m < 16; m <<= 1) v += __shfl_xor(v, m);
      if (j == 0 && has_g) gstore(a.ws_d + at + cg + r, v);
    }
    if (has_j) {
#pragma unroll
      for (int i = 0; i < 4 * M; ++i) gstore(a.ws_h + (at + cj) * N + 4 * g + 16 * (i / 4) + i % 4, st.h[i]);
    }
  } else if (seg == last && has_j) {
#pragma unroll
    for (int i = 0; i < 4 * M; ++i) scan_state_store(a.state, st0 + 16 * (i / 4) + i % 4, a.state_dtype, st.h[i]);
  }
}

// v of lane T of the lane's row of 16.
template <int T>
__device__ __forceinline__ float row_bcast(float v) {
  return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x150 + T, 0xf, 0xf, true));
}

// Pairs of v[t] and v[t + n]: in the lanes of `banks` (groups of 4 in each row of 16) the second, otherwise the first, added
// to its partner lane's (row_ror:8: 8 lanes on; row_half_mirror: 7 - lane of 8).  The leading wait is the broadcast's
// after a vector write.
#define RSSM_PAIR(ctrl, banks)                                                                        \
  asm("s_nop 1\n\tv_add_f32_dpp %0, %1, %1 " ctrl " row_mask:0xf bank_mask:0xf\n\t"                   \
      "v_add_f32_dpp %0, %2, %2 " ctrl " row_mask:0xf bank_mask:" banks                               \
      : "=&v"(o) : "v"(a), "v"(b))
__device__ __forceinline__ float pair_eight(float a, float b) {
  float o;
  RSSM_PAIR("row_ror:8", "0xc");
  return o;
}
__device__ __forceinline__ float pair_four(float a, float b) {
  float o;
  RSSM_PAIR("row_half_mirror", "0xa");
  return o;
}
#undef RSSM_PAIR

template <int CTRL>
__device__ __forceinline__ float quad_add(float v) {
  return v + __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, 0xf, 0xf, true));
}

// Lane j of each row of 16: v[j] summed over the row.
__device__ __forceinline__ float row_sums(const float (&v)[16], int j) {
  float w[8], x[4];
#pragma unroll
  for (int t = 0; t < 8; ++t) w[t] = pair_eight(v[t], v[t + 8]);
#pragma unroll
  for (int t = 0; t < 4; ++t) x[t] = pair_four(w[t], w[t + 4]);
#pragma unroll
  for (int t = 0; t < 4; ++t) x[t] = quad_add<0xB1>(x[t]);   // lane ^ 1; all lanes take part before any is chosen
  const float a = quad_add<0x4E>(j & 1 ? x[1] : x[0]);       // lane ^ 2
  const float b = quad_add<0x4E>(j & 1 ? x[3] : x[2]);
  return j & 2 ? b : a;
}

template <int M, int Q, int T>
__device__ __forceinline__ float scan_short_token(float d, float dx, const f32x4 (&B)[M], const f32x4 (&C)[M],
                                                  const float (&A)[M], float (&h)[M]) {
  float y = 0.0f;
#pragma unroll
  for (int m = 0; m < M; ++m) {
    const float e = __builtin_amdgcn_exp2f(row_bcast<4 * Q + T>(d) * A[m]);
    h[m] = fmaf(e, h[m], row_bcast<4 * Q + T>(dx) * B[m][T]);
    y = m == 0 ? h[0] * C[0][T] : fmaf(h[m], C[m][T], y);
  }
  return y;
}

template <int M, int Q>
__device__ __forceinline__ void scan_short_four(float d, float dx, const float* sB, const float* sC, const float (&A)[M],
                                                float (&h)[M], float (&v)[16]) {
  f32x4 B[M], C[M];
#pragma unroll
  for (int m = 0; m < M; ++m) {
    B[m] = *reinterpret_cast<const f32x4*>(sB + 16 * m * kScanPitch + 4 * Q);
    C[m] = *reinterpret_cast<const f32x4*>(sC + 16 * m * kScanPitch + 4 * Q);
  }
  v[4 * Q] = scan_short_token<M, Q, 0>(d, dx, B, C, A, h);
  v[4 * Q + 1] = scan_short_token<M, Q, 1>(d, dx, B, C, A, h);
  v[4 * Q + 2] = scan_short_token<M, Q, 2>(d, dx, B, C, A, h);
  v[4 * Q + 3] = scan_short_token<M, Q, 3>(d, dx, B, C, A, h);
}

// For few channels and short sequences, where a tile's latency is the time: a wavefront owns 4 channels, lane 16 q + j the
// states j, 16 + j, .. of channel q, a quarter of scan_kernel's work in one lane.  Step sizes and inputs are broadcast from
// the lane of their token; B and C go through LDS to the lanes of their states.  97 tokens of 1,024 channels: 7.0 us, 13.3 by
// scan_kernel; it takes 1.8 times the instructions for each token and channel, which is why the long and wide ones go there.
template <int IT, int N>
__global__ __launch_bounds__(kScanBlock) void scan_short_kernel(ScanArgs a) {
  constexpr int es = sizeof(typename Mma<IT>::elem);
  constexpr int M = N / 16;
  __shared__ alignas(16) float lds[kScanBlock / 64][2][N * kScanPitch];
  const int tid = threadIdx.x, lane = tid & 63, j = lane & 15, q = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int s = blockIdx.x / a.blocks, c0 = (blockIdx.x - s * a.blocks) * kScanShortChannels + 4 * wave;
  if (c0 >= a.channels) return;
  const int slot = sload(a.slots + s);
  if (slot == a.pad || slot < 0 || slot >= a.num_slots) return;
  int start = sload(a.seq_start + s), end = sload(a.seq_start + s + 1);
  start = start < 0 ? 0 : (start > a.num_tokens ? a.num_tokens : start);
  end = end < start ? start : (end > a.num_tokens ? a.num_tokens : end);
  const int n = end - start < a.max_seq_len ? end - start : a.max_seq_len;
  const int c = c0 + q;                                       // channels come in eights: all four are there
  const int gN = a.groups * N;
  ScanRows xr, dr, zr, Br, Cr, yr;
  xr.start(a.x, start, a.x_stride, a.channels * es, es);
  dr.start(a.dt, start, a.dt_stride, a.channels * es, es);
  Br.start(a.B, start, a.B_stride, gN * es, es);
  Cr.start(a.C, start, a.C_stride, gN * es, es);
  yr.start(a.y, start, a.y_stride, a.channels * es, es);
  const bool gated = a.z != nullptr;
  zr.start(gated ? a.z : a.x, start, gated ? a.z_stride : a.x_stride, a.channels * es, es);
  const uint32_t row = static_cast<uint32_t>(c0 / a.per_group) * N;
  const uint32_t xo = j * xr.step + c * es, dto = j * dr.step + c * es, zo = j * zr.step + c * es, yo = j * yr.step + c * es;
  const uint32_t Bo = j * Br.step + (row + 4 * q) * es, Co = j * Cr.step + (row + 4 * q) * es;
  uint32_t rx = 0, rd = 0, rz = 0;
  ScanFour<IT> rB[M], rC[M];
  const auto fetch = [&](int rows) {
    rx = scan_one_load<IT>(xr.tile(rows), xo);
    rd = scan_one_load<IT>(dr.tile(rows), dto);
    rz = scan_one_load<IT>(zr.tile(rows), zo);
    const rsrc_t rb = Br.tile(rows), rc = Cr.tile(rows);
#pragma unroll
    for (int m = 0; m < M; ++m) {
      rB[m].load(rb, Bo + 16 * m * es);
      rC[m].load(rc, Co + 16 * m * es);
    }
    xr.next();
    dr.next();
    zr.next();
    Br.next();
    Cr.next();
  };
  if (n > 0) fetch(n);
  const int64_t st0 = slot * a.state_stride + static_cast<int64_t>(c) * N + j;
  float A[M], h[M];
  const bool load = a.load_state == nullptr || sload(a.load_state + s) != 0;
#pragma unroll
  for (int m = 0; m < M; ++m) {
    A[m] = scan_rate(gload(a.A + static_cast<int64_t>(c) * N + j + 16 * m));
    h[m] = load ? scan_state_load(a.state, st0 + 16 * m, a.state_dtype) : 0.0f;
  }
  const float bias = a.dt_bias != nullptr ? gload(a.dt_bias + c) : 0.0f;
  const float D = a.D != nullptr ? gload(a.D + c) : 0.0f;
  float* const wB = lds[wave][0] + 4 * q * kScanPitch + j;    // token j, states 16 m + 4 q ..
  float* const wC = lds[wave][1] + 4 * q * kScanPitch + j;
  const float* const sB = lds[wave][0] + j * kScanPitch;      // states 16 m + j
  const float* const sC = lds[wave][1] + j * kScanPitch;
  for (int t0 = 0; t0 < n; t0 += kScanTile) {
#pragma unroll
    for (int m = 0; m < M; ++m) {
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        wB[(16 * m + r) * kScanPitch] = rB[m].get(r);
        wC[(16 * m + r) * kScanPitch] = rC[m].get(r);
      }
    }
    const float x = scan_one<IT>(rx), z = scan_one<IT>(rz);
    float d = scan_step_size(scan_one<IT>(rd), bias, a.dt_softplus);
    d = t0 + j < n ? d : 0.0f;
    const float dx = d * x;
    if (t0 + kScanTile < n) fetch(n - t0 - kScanTile);
    scan_wave_sync();
    float v[16];
    scan_short_four<M, 0>(d, dx, sB, sC, A, h, v);
    scan_short_four<M, 1>(d, dx, sB, sC, A, h, v);
    scan_short_four<M, 2>(d, dx, sB, sC, A, h, v);
    scan_short_four<M, 3>(d, dx, sB, sC, A, h, v);
    float y = fmaf(D, x, row_sums(v, j));
    if (gated) y *= silu(z);
    const rsrc_t ry = yr.tile(n - t0);
    if constexpr (IT == kF32) bstore_f32(ry, yo, 0, y);
    else if constexpr (IT == kBF16) __builtin_amdgcn_raw_buffer_store_b16(__builtin_bit_cast(uint16_t, static_cast<__bf16>(y)), ry, yo, 0, 0);
    else __builtin_amdgcn_raw_buffer_store_b16(__builtin_bit_cast(uint16_t, static_cast<_Float16>(y)), ry, yo, 0, 0);
    yr.next();
    scan_wave_sync();
  }
#pragma unroll
  for (int m = 0; m < M; ++m) scan_state_store(a.state, st0 + 16 * m, a.state_dtype, h[m]);
}

// v summed over LPC neighbouring lanes (2 to 16), the same sum in each.
template <int LPC>
__device__ __forceinline__ float lanes_sum(float v) {
  const auto add = [](float x, float y) { return x + y; };
  v = add(v, __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0xB1, 0xf, 0xf, true)));                     // lane ^ 1
  if constexpr (LPC > 2) v = add(v, __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x4E, 0xf, 0xf, true)));   // lane ^ 2
  if constexpr (LPC > 4) v = add(v, __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x141, 0xf, 0xf, true)));  // 7 - lane
  if constexpr (LPC > 8) v = add(v, __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x140, 0xf, 0xf, true)));  // 15 - lane
  return v;
}

// v of the lane of `piece` in the lane's group of R (2 or 4).
template <int R, int PIECE>
__device__ __forceinline__ float piece_bcast(float v) {
  constexpr int ctrl = R == 4 ? PIECE * 0x55 : (PIECE == 0 ? 0xA0 : 0xF5);   // quad_perm
  return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), ctrl, 0xf, 0xf, true));
}

// One piece of a request: the states move on; the lane's part of y.
template <int ST, int EV, int R, int PIECE, typename RawBC>
__device__ __forceinline__ float scan_step_piece(u32x4& raw, float d, float dx, const float* A, const RawBC& B, const RawBC& C) {
  const float dp = piece_bcast<R, PIECE>(d), xp = piece_bcast<R, PIECE>(dx);
  float h[EV], p = 0.0f;
  if constexpr (ST == kF32) {
    const f32x4 v = __builtin_bit_cast(f32x4, raw);
#pragma unroll
    for (int i = 0; i < 4; ++i) h[i] = v[i];
  } else {
    const f32x8 v = from_frag<ST>(__builtin_bit_cast(typename Mma<ST>::frag, raw));
#pragma unroll
    for (int i = 0; i < 8; ++i) h[i] = v[i];
  }
#pragma unroll
  for (int i = 0; i < EV; ++i) {
    h[i] = fmaf(__builtin_amdgcn_exp2f(dp * A[i]), h[i], xp * B.get(i));
    p = fmaf(h[i], C.get(i), p);
  }
  if constexpr (ST == kF32) raw = __builtin_bit_cast(u32x4, f32x4{h[0], h[1], h[2], h[3]});
  else raw = __builtin_bit_cast(u32x4, to_frag<ST>(f32x8{h[0], h[1], h[2], h[3], h[4], h[5], h[6], h[7]}));
  return p;
}

// Q requests a wavefront, which share A, D and bias.  LPC lanes hold a channel's states, 16 bytes each; a wavefront takes R
// pieces of 64 / LPC channels that follow one another.  The step sizes, inputs and outputs of piece r are those of the
// lanes r modulo R: one load, one softplus and one gate a lane for R channels.  256 requests of 8,192 channels, fp16
// with 16 fp32 states: 52 us, 5.5 TB/s, also over pools past the caches in turn (a kilobyte of each of four requests a wavefront instead of four of one: 57 us).
template <int IT, int ST, int N, int Q>
__global__ __launch_bounds__(kScanBlock) void scan_step_kernel(ScanArgs a) {
  typedef typename Mma<IT>::elem elem;
  constexpr int ss = sizeof(typename Mma<ST>::elem), es = sizeof(elem);
  constexpr int EV = 16 / ss;              // states a lane
  constexpr int LPC = N / EV, CPP = 64 / LPC;
  constexpr int R = LPC < 4 ? 2 : 4;
  const int tid = threadIdx.x, lane = tid & 63, part = lane % LPC;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int blk = blockIdx.x % a.blocks, b0 = (blockIdx.x / a.blocks) * Q;
  const int c0 = (blk * (kScanBlock / 64) + wave) * (R * CPP);
  if (c0 >= a.channels) return;
  const int mine = c0 + (lane % R) * CPP + lane / LPC;        // the channel whose input and output are the lane's
  const bool has = mine < a.channels;
  const int cm = has ? mine : c0;
  const int64_t row = static_cast<int64_t>(c0 / a.per_group) * N + part * EV;
  // groups that end inside the wavefront's channels: B and C by piece
  const int c1 = c0 + R * CPP < a.channels ? c0 + R * CPP : a.channels;
  const bool mixed = c0 / a.per_group != (c1 - 1) / a.per_group;
  u32x4 raw[Q][R];
  ScanRaw<IT, EV> rB[Q], rC[Q];
  elem rx[Q], rd[Q], rz[Q];
  char* sp[Q];
#pragma unroll
  for (int q = 0; q < Q; ++q) {
    const int b = b0 + q < a.num_seqs ? b0 + q : a.num_seqs - 1;
    const int slot = sload(a.slots + b);
    const bool live = b0 + q < a.num_seqs && slot != a.pad && slot >= 0 && slot < a.num_slots;
    sp[q] = live ? a.state + (slot * a.state_stride + static_cast<int64_t>(c0) * N + lane * EV) * ss : nullptr;
    if (!live) continue;
#pragma unroll
    for (int r = 0; r < R; ++r)
      if (c0 + r * CPP + lane / LPC < a.channels) raw[q][r] = ld<true, u32x4>(sp[q] + r * 1024);
    rx[q] = gload(reinterpret_cast<const elem*>(a.x) + b * a.x_stride + cm);
    rd[q] = gload(reinterpret_cast<const elem*>(a.dt) + b * a.dt_stride + cm);
    if (a.z != nullptr) rz[q] = gload(reinterpret_cast<const elem*>(a.z) + b * a.z_stride + cm);
    rB[q].load(a.B + (b * a.B_stride + row) * es);
    rC[q].load(a.C + (b * a.C_stride + row) * es);
  }
  float A[R][EV];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int c = c0 + r * CPP + lane / LPC;
    const char* p = reinterpret_cast<const char*>(a.A + static_cast<int64_t>(c < a.channels ? c : c0) * N + part * EV);
#pragma unroll
    for (int k = 0; k < EV / 4; ++k) {
      const f32x4 v = __builtin_bit_cast(f32x4, ld<false, u32x4>(p + 16 * k));
#pragma unroll
      for (int i = 0; i < 4; ++i) A[r][4 * k + i] = scan_rate(v[i]);
    }
  }
  const float bias = a.dt_bias != nullptr ? gload(a.dt_bias + cm) : 0.0f;
  const float D = a.D != nullptr ? gload(a.D + cm) : 0.0f;
#pragma unroll
  for (int q = 0; q < Q; ++q) {
    if (sp[q] == nullptr) continue;        // the same for the whole wavefront
    const float d = scan_step_size(elem_to_float<IT>(rd[q]), bias, a.dt_softplus);
    const float x = elem_to_float<IT>(rx[q]), dx = d * x;
    const auto group = [&](int r) {
      if (!mixed) return;
      const int c = c0 + r * CPP + lane / LPC;
      const int64_t at = static_cast<int64_t>((c < a.channels ? c : c0) / a.per_group) * N + part * EV;
      rB[q].load(a.B + ((b0 + q) * a.B_stride + at) * es);
      rC[q].load(a.C + ((b0 + q) * a.C_stride + at) * es);
    };
    float p[R];
    group(0);
    p[0] = lanes_sum<LPC>(scan_step_piece<ST, EV, R, 0>(raw[q][0], d, dx, A[0], rB[q], rC[q]));
    group(1);
    p[1] = lanes_sum<LPC>(scan_step_piece<ST, EV, R, 1>(raw[q][1], d, dx, A[1], rB[q], rC[q]));
    if constexpr (R == 4) {
      group(2);
      p[2] = lanes_sum<LPC>(scan_step_piece<ST, EV, R, 2>(raw[q][2], d, dx, A[2], rB[q], rC[q]));
      group(3);
      p[3] = lanes_sum<LPC>(scan_step_piece<ST, EV, R, 3>(raw[q][3], d, dx, A[3], rB[q], rC[q]));
    }
#pragma unroll
    for (int r = 0; r < R; ++r)
      if (c0 + r * CPP + lane / LPC < a.channels) st<true>(sp[q] + r * 1024, raw[q][r]);
    float y = lane & 1 ? p[1] : p[0];
    if constexpr (R == 4) y = lane & 2 ? (lane & 1 ? p[3] : p[2]) : y;
    y = fmaf(D, x, y);
    if (a.z != nullptr) y *= silu(elem_to_float<IT>(rz[q]));
    if (has && part < R) {
      elem* yp = reinterpret_cast<elem*>(a.y) + (b0 + q) * a.y_stride + mine;
      if constexpr (IT == kF32) gstore(yp, y);
      else if constexpr (IT == kBF16) gstore(yp, __builtin_bit_cast(uint16_t, static_cast<__bf16>(y)));
      else gstore(yp, __builtin_bit_cast(uint16_t, static_cast<_Float16>(y)));
    }
  }
}

}  // namespace rssm
