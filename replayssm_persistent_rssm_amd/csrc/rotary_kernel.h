// rotary_kernel.h -- gfx950 kernel of rotary positions with the append to a paged cache.
//
// A wavefront takes one token and a share of its heads.  The angles of a token are the same for all its heads: lane i
// computes the sine and cosine of pair i (position times frequency, and its remainder modulo a turn, in 64
// bits), and every lane picks the eight pairs it turns through LDS.  A lane's unit is two vectors of 8
// elements of a head that hold 8 whole pairs: vectors 2u and 2u + 1 when interleaved, vectors u and
// u + rot_dim / 16 otherwise; units past rot_dim pass through.  Few tokens are shared out over up to 8 wavefronts each.  Bound
// by memory: 18,900 ragged fp16 tokens of 32 + 2 x 8 heads of 128: 95 us, 4.9 TB/s, the rate of a large copy (past the caches
// 138 us); a decoding batch of 64 tokens by the launch, 4.1 us.
#pragma once

#include "mma_device.h"

namespace rssm {

struct RotaryArgs {
  const char* q;
  char* q_out;
  const char* k_new;
  const char* v_new;
  char* k;
  char* v;
  const int32_t* table;
  const int32_t* seq_start;   // or null
  const int32_t* kv_len;
  const int32_t* positions;   // or null
  const float* inv_freq;
  int64_t page_stride, row_stride, head_stride, q_stride, qo_stride, k_stride, v_stride, table_stride;   // elements
  int32_t num_seqs, num_tokens, Hq, Hkv, rot_dim, interleaved, page_size, num_pages, max_pages;
  float factor;
  int32_t shares;             // wavefronts a token
  int32_t units;              // num_tokens * shares
};

constexpr int kRotaryBlock = 256;

// Sequence of row `token`: the first that ends after it (num_seqs if none), uniform over the wavefront.  The last 64
// candidates are asked at once.
__device__ __forceinline__ int rotary_seq(const RotaryArgs& a, int token, int lane) {
  int lo = 0, hi = a.num_seqs;
  while (hi - lo > 64) {
    const int mid = (lo + hi) >> 1;
    if (sload(a.seq_start + mid + 1) > token) hi = mid;
    else lo = mid + 1;
  }
  const int i = lo + lane;
  const bool past = i < hi && gload(a.seq_start + i + 1) <= token;
  return lo + __builtin_popcountll(__ballot(past));
}

// Sine and cosine of p f, f in radians a position: the turns p f / (2 pi) in 64 bits, their part in [-1/2, 1/2] to fp32.
__device__ __forceinline__ void rotary_angle(int p, float f, float factor, float& c, float& s) {
  double turns = static_cast<double>(p) * static_cast<double>(f) * 0.15915494309189533577;
  turns -= __builtin_rint(turns);
  sincospif(2.0f * static_cast<float>(turns), &s, &c);
  c *= factor;
  s *= factor;
}

// Eight elements in storage.
template <int DT>
struct Eight {
  static constexpr int kParts = sizeof(typename Mma<DT>::elem) / 2;
  u32x4 v[kParts];
  __device__ __forceinline__ void load(const char* p) {
#pragma unroll
    for (int k = 0; k < kParts; ++k) v[k] = ld<false, u32x4>(p + 16 * k);
  }
  __device__ __forceinline__ void store(char* p) const {
#pragma unroll
    for (int k = 0; k < kParts; ++k) st<false>(p + 16 * k, v[k]);
  }
  __device__ __forceinline__ f32x8 get() const {
    if constexpr (DT == kF32) return stack(__builtin_bit_cast(f32x4, v[0]), __builtin_bit_cast(f32x4, v[1]));
    else return from_frag<DT>(__builtin_bit_cast(typename Mma<DT>::frag, v[0]));
  }
  __device__ __forceinline__ void set(f32x8 x) {
    if constexpr (DT == kF32) {
      v[0] = __builtin_bit_cast(u32x4, f32x4{x[0], x[1], x[2], x[3]});
      v[1] = __builtin_bit_cast(u32x4, f32x4{x[4], x[5], x[6], x[7]});
    } else {
      v[0] = __builtin_bit_cast(u32x4, to_frag<DT>(x));
    }
  }
};

template <int DT, int D>
__global__ __launch_bounds__(kRotaryBlock) void rotary_kernel(RotaryArgs a) {
  constexpr int es = sizeof(typename Mma<DT>::elem);
  constexpr int U = D / 16;              // units a head
  constexpr int HP = 64 / U;             // heads a pass
  __shared__ alignas(16) float lds[kRotaryBlock / 64][2][64];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int unit = blockIdx.x * (kRotaryBlock / 64) + wave;
  if (unit >= a.units) return;
  const int token = unit / a.shares, share = unit - token * a.shares;
  // place in the cache (negative or past the last: none)
  int64_t place = -1;
  int s = 0;
  if (a.seq_start != nullptr) {
    s = __builtin_amdgcn_readfirstlane(rotary_seq(a, token, lane));
    if (s >= a.num_seqs) return;
    const int start = sload(a.seq_start + s), end = sload(a.seq_start + s + 1);
    if (token < start) return;
    if (a.kv_len != nullptr) place = static_cast<int64_t>(sload(a.kv_len + s)) - (end < a.num_tokens ? end : a.num_tokens) + token;
  }
  const int pos = a.positions != nullptr ? sload(a.positions + token) : static_cast<int>(place);
  int64_t row = -1;                      // of head 0 in the caches, in elements; -1: not appended
  if (a.Hkv > 0 && place >= 0 && place < static_cast<int64_t>(a.max_pages) * a.page_size) {
    const int pi = static_cast<int>(place / a.page_size);
    const int page = sload(a.table + s * a.table_stride + pi);
    if (page >= 0 && page < a.num_pages) row = page * a.page_stride + (place - static_cast<int64_t>(pi) * a.page_size) * a.row_stride;
  }
  const int half = a.rot_dim / 2;
  float cs = 0.0f, sn = 0.0f;
  if (lane < half) rotary_angle(pos, gload(a.inv_freq + lane), a.factor, cs, sn);
  lds[wave][0][lane] = cs;
  lds[wave][1][lane] = sn;
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
  const int u = lane % U, rot_units = a.rot_dim / 16;
  const bool turn = u < rot_units;
  // first and second vector of the unit
  const int v0 = turn && !a.interleaved ? u : 2 * u;
  const int v1 = turn && !a.interleaved ? u + rot_units : 2 * u + 1;
  f32x8 c8, s8;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    c8[e] = turn ? lds[wave][0][8 * u + e] : 1.0f;
    s8[e] = turn ? lds[wave][1][8 * u + e] : 0.0f;
  }
  const auto turned = [&](f32x8& x, f32x8& y) {
    if (a.interleaved) {
      const f32x8 p = x, q = y;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        x[2 * e] = fmaf(p[2 * e], c8[e], -p[2 * e + 1] * s8[e]);
        x[2 * e + 1] = fmaf(p[2 * e], s8[e], p[2 * e + 1] * c8[e]);
        y[2 * e] = fmaf(q[2 * e], c8[4 + e], -q[2 * e + 1] * s8[4 + e]);
        y[2 * e + 1] = fmaf(q[2 * e], s8[4 + e], q[2 * e + 1] * c8[4 + e]);
      }
    } else {
      const f32x8 p = x, q = y;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        x[e] = fmaf(p[e], c8[e], -q[e] * s8[e]);
        y[e] = fmaf(p[e], s8[e], q[e] * c8[e]);
      }
    }
  };
  const int total = a.Hq + (row >= 0 ? 2 * a.Hkv : 0);
  for (int h = share * HP + lane / U; h < total; h += a.shares * HP) {
    const char* src;
    char* dst;
    const bool value = h >= a.Hq + a.Hkv;
    if (h < a.Hq) {
      src = a.q + (token * a.q_stride + static_cast<int64_t>(h) * D) * es;
      dst = a.q_out + (token * a.qo_stride + static_cast<int64_t>(h) * D) * es;
    } else {
      const int kh = value ? h - a.Hq - a.Hkv : h - a.Hq;
      src = (value ? a.v_new + token * a.v_stride * es : a.k_new + token * a.k_stride * es) + static_cast<int64_t>(kh) * D * es;
      dst = (value ? a.v : a.k) + (row + kh * a.head_stride) * es;
    }
    Eight<DT> x, y;
    x.load(src + v0 * 8 * es);
    y.load(src + v1 * 8 * es);
    if (turn && !value) {   // what is not turned keeps its bits (a conversion and back would make a signalling NaN a quiet one)
      f32x8 p = x.get(), q = y.get();
      turned(p, q);
      x.set(p);
      y.set(q);
    }
    x.store(dst + v0 * 8 * es);
    y.store(dst + v1 * 8 * es);
  }
}

}  // namespace rssm
