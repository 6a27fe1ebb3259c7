// conv_kernel.h -- gfx950 kernels of the short causal convolution: ragged
// prompts and single tokens.
//
// Both are bound by memory (2 W flops an output of 2 to 4 bytes in and out).  A lane owns 8 channels
// (16 or 32 bytes a row) with their weights in registers.
//  * conv_prompt_kernel: a wavefront walks a tile of consecutive tokens of one sequence over 512 channels,
//    the last W - 1 inputs in registers, so that each input is read once apart from the W - 1 rows before a
//    tile.  Sequence s owns the tiles first_tile(s) .. first_tile(s + 1) - 1 with
//    first_tile(s) = floor(start_s / T) + s: at least ceil(length / T) of them whatever the lengths, without a
//    prefix sum and without knowing the longest sequence.  The state is read and written by a sequence's first tile
//    alone (tiles are longer than W - 1 tokens), so no other wavefront sees it change.  12 ragged prompts up to 2,011
//    tokens, 18,432 bf16 channels (a gigabyte): 192 us, 5.3 TB/s, above the rate of a large copy (4.9) on the same card; with loads
//    and stores past the caches 3% faster alone, but then the kernel that reads y next finds none of it.
//  * conv_step_kernel: a lane takes the same channels of several requests, so that the weights
//    (4 W bytes a channel, as much as a request's own traffic) are read once for them.  256 requests of 18,432 bf16
//    channels: 13.8 us, 5.5 TB/s with the 47 MB of its tensors in the last cache, 22.0 over sets of them past it in turn (a plain
//    copy of as many bytes: 11.3 and 16.2); loads and stores that go past the caches 17.2 in the first case.
#pragma once

#include "mma_device.h"

namespace rssm {

struct ConvArgs {
  const char* x;
  const float* weight;
  const float* bias;          // or null
  char* y;
  char* state;
  const int32_t* slots;
  const int32_t* seq_start;
  const int32_t* load_state;  // or null
  int64_t state_stride, x_stride, y_stride;   // elements
  int32_t num_seqs, num_tokens, channels, num_slots, pad, silu;
  int32_t blocks;             // channel blocks of 512
  int32_t units;              // (tile or request group, channel block) pairs
};

constexpr int kConvBlock = 256;
constexpr int kConvLanes = 64 * 8;   // channels a wavefront

__device__ __forceinline__ int conv_clamp(int v, int hi) { return v < 0 ? 0 : (v > hi ? hi : v); }

// Sequence of tile `tile` (the last one whose first tile is not past it), by a binary search over seq_start;
// uniform over the wavefront.
template <int T>
__device__ __forceinline__ int conv_seq_of(const ConvArgs& a, int tile) {
  int lo = 0, hi = a.num_seqs - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (conv_clamp(sload(a.seq_start + mid), a.num_tokens) / T + mid <= tile) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

template <int DT, int W>
struct ConvWeights {
  f32x8 w[W], b;
  __device__ __forceinline__ ConvWeights(const ConvArgs& a, int c) {
#pragma unroll
    for (int k = 0; k < W; ++k)
      w[k] = load8<kF32>(reinterpret_cast<const char*>(a.weight + static_cast<int64_t>(k) * a.channels + c));
    b = a.bias != nullptr ? load8<kF32>(reinterpret_cast<const char*>(a.bias + c)) : f32x8{0, 0, 0, 0, 0, 0, 0, 0};
  }
};

__device__ __forceinline__ f32x8 conv_act(f32x8 v, int act) {
  if (act) {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = silu(v[e]);
  }
  return v;
}

// Eight elements in storage.
template <int DT> struct Raw8 { u32x4 v; };
template <> struct Raw8<kF32> { u32x4 v, u; };

template <int DT>
__device__ __forceinline__ Raw8<DT> raw_load(const char* p) {
  Raw8<DT> r;
  r.v = ld<false, u32x4>(p);
  if constexpr (DT == kF32) r.u = ld<false, u32x4>(p + 16);
  return r;
}

template <int DT>
__device__ __forceinline__ void raw_store(char* p, Raw8<DT> r) {
  st<false>(p, r.v);
  if constexpr (DT == kF32) st<false>(p + 16, r.u);
}

template <int DT>
__device__ __forceinline__ Raw8<DT> raw_zero() {
  Raw8<DT> r;
  r.v = u32x4{0, 0, 0, 0};
  if constexpr (DT == kF32) r.u = u32x4{0, 0, 0, 0};
  return r;
}

template <int DT>
__device__ __forceinline__ f32x8 raw_float(Raw8<DT> r) {
  if constexpr (DT == kF32) return stack(__builtin_bit_cast(f32x4, r.v), __builtin_bit_cast(f32x4, r.u));
  else return from_frag<DT>(__builtin_bit_cast(typename Mma<DT>::frag, r.v));
}

template <int DT, int W, int T>
__global__ __launch_bounds__(kConvBlock) void conv_prompt_kernel(ConvArgs a) {
  constexpr int es = sizeof(typename Mma<DT>::elem);
  constexpr int kAhead = T < 8 ? T : 8;   // inputs in flight
  static_assert(T % kAhead == 0 && T >= W, "");
  const int lane = threadIdx.x & 63;
  const int unit = __builtin_amdgcn_readfirstlane(xcd_order(blockIdx.x, gridDim.x) * (kConvBlock / 64) + (threadIdx.x >> 6));
  if (unit >= a.units) return;
  const int tile = unit / a.blocks, c = (unit - tile * a.blocks) * kConvLanes + lane * 8;
  const int s = conv_seq_of<T>(a, tile);
  const int start = conv_clamp(sload(a.seq_start + s), a.num_tokens);
  int end = conv_clamp(sload(a.seq_start + s + 1), a.num_tokens);
  end = end < start ? start : end;
  const int slot = sload(a.slots + s);
  const int64_t t0 = start + static_cast<int64_t>(tile - (start / T + s)) * T;
  if (t0 < start || slot == a.pad || slot < 0 || slot >= a.num_slots || c >= a.channels) return;
  if (t0 > start && t0 >= end) return;
  const ConvWeights<DT, W> w(a, c);
  const char* xp = a.x + c * es;
  const int64_t xs = a.x_stride * es;
  const int n = static_cast<int>(end - t0 < T ? end - t0 : T);
  Raw8<DT> hist[W - 1], tail[W - 1];   // the W - 1 inputs before t0 and the sequence's last ones, oldest first
  char* const sp = a.state + (slot * a.state_stride + c) * es;
  const int64_t srow = static_cast<int64_t>(a.channels) * es;
  const bool opens = t0 == start;
  if (opens) {
    const bool load = a.load_state == nullptr || sload(a.load_state + s) != 0;
#pragma unroll
    for (int k = 0; k < W - 1; ++k) hist[k] = load ? raw_load<DT>(sp + k * srow) : raw_zero<DT>();
#pragma unroll
    for (int k = 0; k < W - 1; ++k) {
      const int p = end - start - (W - 1) + k;   // place in the sequence; below 0: hist[p + W - 1]
      tail[k] = raw_zero<DT>();
      if (p >= 0) tail[k] = raw_load<DT>(xp + (start + static_cast<int64_t>(p)) * xs);
    }
  } else {
#pragma unroll
    for (int k = 0; k < W - 1; ++k) hist[k] = raw_load<DT>(xp + (t0 - (W - 1) + k) * xs);
  }
  xp += t0 * xs;
  char* yp = a.y + t0 * a.y_stride * es + c * es;
  const int64_t ys = a.y_stride * es;
  Raw8<DT> in[kAhead];
  const auto fetch = [&](int t) {
#pragma unroll
    for (int i = 0; i < kAhead; ++i) in[i] = raw_load<DT>(xp + (t + i < n ? t + i : n - 1) * xs);
  };
  if (n > 0) fetch(0);
  f32x8 h[W - 1];
#pragma unroll
  for (int k = 0; k < W - 1; ++k) h[k] = raw_float<DT>(hist[k]);
  for (int t = 0; t < n; t += kAhead) {
    if (t > 0) fetch(t);
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      if (t + i < n) {
        const f32x8 v = raw_float<DT>(in[i]);
        f32x8 o = w.b;
#pragma unroll
        for (int k = 0; k < W - 1; ++k) {
#pragma unroll
          for (int e = 0; e < 8; ++e) o[e] = fmaf(w.w[k][e], h[k][e], o[e]);
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) o[e] = fmaf(w.w[W - 1][e], v[e], o[e]);
#pragma unroll
        for (int k = 0; k + 1 < W - 1; ++k) h[k] = h[k + 1];
        h[W - 2] = v;
        store8<DT>(yp + (t + i) * ys, conv_act(o, a.silu));
      }
    }
  }
  if (opens) {   // of a sequence shorter than W - 1, old rows move up
    const int len = end - start;
#pragma unroll
    for (int k = 0; k < W - 1; ++k) {
      Raw8<DT> v = tail[k];
#pragma unroll
      for (int m = k + 1; m < W - 1; ++m)
        if (m == len + k) v = hist[m];
      if (len == 0) v = hist[k];
      raw_store<DT>(sp + k * srow, v);
    }
  }
}

// R requests a lane.
template <int DT, int W, int R>
__global__ __launch_bounds__(kConvBlock) void conv_step_kernel(ConvArgs a) {
  constexpr int es = sizeof(typename Mma<DT>::elem);
  const int lane = threadIdx.x & 63;
  const int unit = __builtin_amdgcn_readfirstlane(blockIdx.x * (kConvBlock / 64) + (threadIdx.x >> 6));
  if (unit >= a.units) return;
  const int group = unit / a.blocks, c = (unit - group * a.blocks) * kConvLanes + lane * 8;
  if (c >= a.channels) return;
  const int64_t row = static_cast<int64_t>(a.channels) * es;
  Raw8<DT> hist[R][W - 1], in[R];
  char* sp[R];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int b = group * R + r;
    const int slot = b < a.num_seqs ? sload(a.slots + b) : a.pad;
    const bool live = b < a.num_seqs && slot != a.pad && slot >= 0 && slot < a.num_slots;
    sp[r] = live ? a.state + (slot * a.state_stride + c) * es : nullptr;
    if (live) {
      in[r] = raw_load<DT>(a.x + (b * a.x_stride + c) * es);
#pragma unroll
      for (int k = 0; k < W - 1; ++k) hist[r][k] = raw_load<DT>(sp[r] + k * row);
    }
  }
  const ConvWeights<DT, W> w(a, c);
#pragma unroll
  for (int r = 0; r < R; ++r) {
    if (sp[r] == nullptr) continue;
    f32x8 o = w.b;
#pragma unroll
    for (int k = 0; k < W; ++k) {
      const f32x8 v = raw_float<DT>(k < W - 1 ? hist[r][k] : in[r]);
#pragma unroll
      for (int e = 0; e < 8; ++e) o[e] = fmaf(w.w[k][e], v[e], o[e]);
    }
#pragma unroll
    for (int k = 0; k < W - 1; ++k) raw_store<DT>(sp[r] + k * row, k + 1 < W - 1 ? hist[r][k + 1] : in[r]);
    store8<DT>(a.y + ((group * R + r) * a.y_stride + c) * es, conv_act(o, a.silu));
  }
}

}  // namespace rssm
