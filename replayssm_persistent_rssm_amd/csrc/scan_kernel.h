// scan_kernel.h -- gfx950 kernels of the selective state-space scan: ragged
// prompts and single tokens.
//
// The decay of each (token, channel, state) is an exponential of its own, so no matrix product does this
// work: one exponential, two products and two multiply-adds for each of them on the vector ALUs are the
// bound, and everything else is arranged so as not to add to it.
//
// scan_kernel: a wavefront owns 16 channels of a sequence and all their states in registers: lane 16 g + j
// has states g N/4 .. (g + 1) N/4 - 1 of channel j.  It walks the tokens in tiles of 16.
//  * Inputs of a tile come as lane 16 g + j = token j, channels 4g .. 4g + 3 (x, dt, z) and token j, states of
//    group g (B, C): one load an input, each step size computed once.
//  * Step sizes go to the channels' lanes through LDS (16 x 16 floats of the wavefront's own, no barrier).
//  * B_t and C_t are the same for all 16 channels: the product's operand is broadcast from lane t of each row of 16
//    by the instruction that uses it (row broadcast), at no cost.
//  * The sums over the four groups of states are taken for four tokens at once by swapping halves and rows of lanes
//    (6 instructions for 4 tokens), and go back to the tile's layout through LDS for skip, gate and store.
// When sequences and channels leave compute units empty, the token axis is split: scan_kernel<FOLD> gives
// each stretch's own end state and the sum of its step sizes (a decay over the stretch is exp(A sum)), and
// the main kernel starts each stretch from those of the stretches before it.
// scan_step_kernel: a lane has 16 bytes of a channel's states; bound by reading and writing the state.
#pragma once

#include <utility>

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
  float* ws_h;                // [num_seqs][nseg][channels][N] (nseg > 1)
  float* ws_d;                // [num_seqs][nseg][channels]
  int64_t state_stride, x_stride, dt_stride, B_stride, C_stride, z_stride, y_stride;   // elements
  int32_t num_seqs, num_tokens, channels, per_group, num_slots, pad, max_seq_len, dt_softplus, state_dtype;
  int32_t nseg, seg_len;      // stretches of the token axis and their length (a multiple of 16)
  int32_t blocks;             // channel blocks
};

constexpr int kScanBlock = 256;
constexpr int kScanChannels = 64;    // a workgroup of scan_kernel, 16 a wavefront
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
  __device__ __forceinline__ void keep(bool on) {
#pragma unroll
    for (int k = 0; k < kWords; ++k) w[k] = on ? w[k] : 0u;
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

// v of lane T of the lane's row of 16.
template <int T>
__device__ __forceinline__ float row_bcast(float v) {
  return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x150 + T, 0xf, 0xf, true));
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

// A log2(e), with -infinity as the most negative number: a step of size 0 then decays by exp2(-0) = 1.
__device__ __forceinline__ float scan_rate(float A) { return fmaxf(A * kLog2e, -3.40282347e38f); }

template <int NS>
struct ScanTile {
  float dt[kScanTile], dx[kScanTile];   // of the lane's channel
  float B[NS], C[NS];                   // of token lane % 16, the lane's group of states
};

// Tokens T .. of a tile: the states move on, p[t] is the lane's part of y_t.
template <int NS, bool FOLD, int T>
__device__ __forceinline__ float scan_token(const ScanTile<NS>& k, const float (&A)[NS], float (&h)[NS]) {
  float p = 0.0f;
#pragma unroll
  for (int i = 0; i < NS; ++i) {
    const float e = __builtin_amdgcn_exp2f(k.dt[T] * A[i]);
    h[i] = fmaf(e, h[i], row_bcast<T>(k.B[i]) * k.dx[T]);
  }
  if constexpr (!FOLD) {
    p = scan_dot4<T, true>(p, k.C, h);
#pragma unroll
    for (int i = 4; i < NS; i += 4) p = scan_dot4<T, false>(p, k.C + i, h + i);
  }
  return p;
}

template <int NS, bool FOLD, int Q>
__device__ __forceinline__ float scan_four(const ScanTile<NS>& k, const float (&A)[NS], float (&h)[NS]) {
  const float p0 = scan_token<NS, FOLD, 4 * Q>(k, A, h);
  const float p1 = scan_token<NS, FOLD, 4 * Q + 1>(k, A, h);
  const float p2 = scan_token<NS, FOLD, 4 * Q + 2>(k, A, h);
  const float p3 = scan_token<NS, FOLD, 4 * Q + 3>(k, A, h);
  if constexpr (FOLD) return 0.0f;
  return rows_sum(halves_sum(p0, p2), halves_sum(p1, p3));   // row g: token 4 Q + g
}

template <int IT, int N, bool FOLD>
__global__ __launch_bounds__(kScanBlock) void scan_kernel(ScanArgs a) {
  constexpr int es = sizeof(typename Mma<IT>::elem);
  constexpr int NS = N / 4;
  __shared__ alignas(16) float lds[kScanBlock / 64][3][kScanTile * kScanPitch];
  const int tid = threadIdx.x, lane = tid & 63, j = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  int u = blockIdx.x;
  const int c0 = (u % a.blocks) * kScanChannels + wave * 16;
  u /= a.blocks;
  const int seg = u % a.nseg, s = u / a.nseg;
  const int slot = sload(a.slots + s);
  if (slot == a.pad || slot < 0 || slot >= a.num_slots || c0 >= a.channels) return;
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
  const int64_t st0 = slot * a.state_stride + static_cast<int64_t>(cj) * N + g * NS;
  float A[NS], h[NS];
#pragma unroll
  for (int i = 0; i < NS; ++i) {
    A[i] = has_j ? scan_rate(gload(a.A + static_cast<int64_t>(cj) * N + g * NS + i)) : 0.0f;
    h[i] = 0.0f;
  }
  if (!FOLD && has_j) {
    if (a.load_state == nullptr || sload(a.load_state + s) != 0) {
#pragma unroll
      for (int i = 0; i < NS; ++i) h[i] = scan_state_load(a.state, st0 + i, a.state_dtype);
    }
    for (int k = 0; k < seg; ++k) {
      const int64_t at = (static_cast<int64_t>(s) * a.nseg + k) * a.channels + cj;
      const float sum = gload(a.ws_d + at);
#pragma unroll
      for (int i = 0; i < NS; ++i)
        h[i] = fmaf(__builtin_amdgcn_exp2f(sum * A[i]), h[i], gload(a.ws_h + at * N + g * NS + i));
    }
  }
  float bias[4], D[4], dsum[4] = {0, 0, 0, 0};
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    bias[r] = a.dt_bias != nullptr && has_g ? gload(a.dt_bias + cg + r) : 0.0f;
    D[r] = a.D != nullptr && has_g ? gload(a.D + cg + r) : 0.0f;
  }
  // rows of the lane's token and of the first tile; channels past the end read channel block c0
  const int col = has_g ? cg : c0;
  const int64_t row = static_cast<int64_t>(c0 / a.per_group) * N + g * NS;
  const char* xp = a.x + (tok * a.x_stride + col) * es;
  const char* dp = a.dt + (tok * a.dt_stride + col) * es;
  const char* zp = a.z != nullptr ? a.z + (tok * a.z_stride + col) * es : nullptr;
  const char* Bp = a.B + (tok * a.B_stride + row) * es;
  const char* Cp = a.C + (tok * a.C_stride + row) * es;
  char* yp = a.y + (tok * a.y_stride + col) * es;
  ScanRaw<IT, 4> rx, rd, rz;
  ScanRaw<IT, NS> rB, rC;
  rz.keep(false);
  const auto fetch = [&](int t0) {
    const int64_t t = t0 + j < n ? t0 + j : n - 1;
    rx.load(xp + t * a.x_stride * es);
    rd.load(dp + t * a.dt_stride * es);
    rB.load(Bp + t * a.B_stride * es);
    if constexpr (!FOLD) {
      rC.load(Cp + t * a.C_stride * es);
      if (zp != nullptr) rz.load(zp + t * a.z_stride * es);
    }
  };
  if (n > 0) fetch(0);
  float* const sd = lds[wave][0];
  float* const sx = lds[wave][1];
  float* const sy = lds[wave][2];
  for (int t0 = 0; t0 < n; t0 += kScanTile) {
    const bool on = t0 + j < n;
    ScanTile<NS> k;
    float x[4], z[4];
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      x[r] = on && has_g ? rx.get(r) : 0.0f;
      z[r] = rz.get(r);
      float d = prompt_dt(rd.get(r), bias[r], a.dt_softplus);
      d = on && has_g ? d : 0.0f;
      if constexpr (FOLD) dsum[r] += d;
      sd[(4 * g + r) * kScanPitch + j] = d;
      sx[(4 * g + r) * kScanPitch + j] = d * x[r];
    }
    rB.keep(on);
    if constexpr (!FOLD) rC.keep(on);
#pragma unroll
    for (int i = 0; i < NS; ++i) {
      k.B[i] = rB.get(i);
      k.C[i] = FOLD ? 0.0f : rC.get(i);
    }
    if (t0 + kScanTile < n) fetch(t0 + kScanTile);
    scan_wave_sync();
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const f32x4 d = *reinterpret_cast<const f32x4*>(sd + j * kScanPitch + 4 * q);
      const f32x4 v = *reinterpret_cast<const f32x4*>(sx + j * kScanPitch + 4 * q);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        k.dt[4 * q + e] = d[e];
        k.dx[4 * q + e] = v[e];
      }
    }
    const float y0 = scan_four<NS, FOLD, 0>(k, A, h);
    const float y1 = scan_four<NS, FOLD, 1>(k, A, h);
    const float y2 = scan_four<NS, FOLD, 2>(k, A, h);
    const float y3 = scan_four<NS, FOLD, 3>(k, A, h);
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
        if (zp != nullptr) y[r] *= silu(z[r]);
      }
      if (on && has_g) narrow4<IT>(reinterpret_cast<typename Mma<IT>::elem*>(yp + (t0 + j) * a.y_stride * es), y);
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
      for (int i = 0; i < NS; ++i) gstore(a.ws_h + (at + cj) * N + g * NS + i, h[i]);
    }
  } else if (seg == last && has_j) {
#pragma unroll
    for (int i = 0; i < NS; ++i) scan_state_store(a.state, st0 + i, a.state_dtype, h[i]);
  }
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

// R requests a lane share the channel's A, D and bias.
template <int IT, int ST, int N, int R>
__global__ __launch_bounds__(kScanBlock) void scan_step_kernel(ScanArgs a) {
  typedef typename Mma<IT>::elem elem;
  constexpr int ss = sizeof(typename Mma<ST>::elem), es = sizeof(elem);
  constexpr int EV = 16 / ss;              // states a lane
  constexpr int LPC = N / EV;              // lanes a channel
  const int tid = threadIdx.x, part = tid % LPC;
  const int blk = blockIdx.x % a.blocks, b0 = (blockIdx.x / a.blocks) * R;
  const int c = blk * (kScanBlock / LPC) + tid / LPC;
  const bool has = c < a.channels;         // all lanes stay for the sums
  const int cc = has ? c : 0;
  u32x4 raw[R];
  ScanRaw<IT, EV> rB[R], rC[R];
  elem rx[R], rd[R], rz[R];
  char* sp[R];
  const int64_t row = static_cast<int64_t>(cc / a.per_group) * N + part * EV;
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int b = b0 + r < a.num_seqs ? b0 + r : a.num_seqs - 1;
    const int slot = sload(a.slots + b);
    const bool live = b0 + r < a.num_seqs && slot != a.pad && slot >= 0 && slot < a.num_slots;
    sp[r] = live ? a.state + (slot * a.state_stride + static_cast<int64_t>(cc) * N + part * EV) * ss : nullptr;
    if (!live) continue;
    raw[r] = ld<true, u32x4>(sp[r]);
    rB[r].load(a.B + (b * a.B_stride + row) * es);
    rC[r].load(a.C + (b * a.C_stride + row) * es);
    rx[r] = gload(reinterpret_cast<const elem*>(a.x) + b * a.x_stride + cc);
    rd[r] = gload(reinterpret_cast<const elem*>(a.dt) + b * a.dt_stride + cc);
    if (a.z != nullptr) rz[r] = gload(reinterpret_cast<const elem*>(a.z) + b * a.z_stride + cc);
  }
  f32x4 A[EV / 4];
#pragma unroll
  for (int k = 0; k < EV / 4; ++k)
    A[k] = __builtin_bit_cast(f32x4, ld<false, u32x4>(reinterpret_cast<const char*>(a.A + static_cast<int64_t>(cc) * N + part * EV + 4 * k)));
  const float bias = a.dt_bias != nullptr ? gload(a.dt_bias + cc) : 0.0f;
  const float D = a.D != nullptr ? gload(a.D + cc) : 0.0f;
#pragma unroll
  for (int r = 0; r < R; ++r) {
    if (sp[r] == nullptr) continue;        // the same for the whole wavefront
    const float d = prompt_dt(elem_to_float<IT>(rd[r]), bias, a.dt_softplus);
    const float x = elem_to_float<IT>(rx[r]), dx = d * x;
    float h[EV], p = 0.0f;
    if constexpr (ST == kF32) {
      const f32x4 v = __builtin_bit_cast(f32x4, raw[r]);
#pragma unroll
      for (int i = 0; i < 4; ++i) h[i] = v[i];
    } else {
      const f32x8 v = from_frag<ST>(__builtin_bit_cast(typename Mma<ST>::frag, raw[r]));
#pragma unroll
      for (int i = 0; i < 8; ++i) h[i] = v[i];
    }
#pragma unroll
    for (int i = 0; i < EV; ++i) {
      const float e = __builtin_amdgcn_exp2f(d * scan_rate(A[i / 4][i % 4]));
      h[i] = fmaf(e, h[i], dx * rB[r].get(i));
      p = fmaf(h[i], rC[r].get(i), p);
    }
    p = lanes_sum<LPC>(p);
    if (!has) continue;
    u32x4 o;
    if constexpr (ST == kF32) {
      o = __builtin_bit_cast(u32x4, f32x4{h[0], h[1], h[2], h[3]});
    } else {
      o = __builtin_bit_cast(u32x4, to_frag<ST>(f32x8{h[0], h[1], h[2], h[3], h[4], h[5], h[6], h[7]}));
    }
    st<true>(sp[r], o);
    if (part == 0) {
      float y = fmaf(D, x, p);
      if (a.z != nullptr) y *= silu(elem_to_float<IT>(rz[r]));
      elem* yp = reinterpret_cast<elem*>(a.y) + (b0 + r) * a.y_stride + c;
      if constexpr (IT == kF32) gstore(yp, y);
      else if constexpr (IT == kBF16) gstore(yp, __builtin_bit_cast(uint16_t, static_cast<__bf16>(y)));
      else gstore(yp, __builtin_bit_cast(uint16_t, static_cast<_Float16>(y)));
    }
  }
}

}  // namespace rssm
