// norm_kernel.h -- gfx950 kernel of the norms around a block: gate, grouped
// norm of the block's output, scaled addition to the residual, norm before the
// next block.
//
// One workgroup a row; the row stays in registers (VPT vectors of 8 channels a
// thread), so each tensor is read or written once.  Sums of squares go lane -> wavefront
// (shuffles) -> LDS in a fixed order.  16,384 rows of 8,192 channels, bf16 with an fp32 residual: 0.338 ms,
// 4.8 TB/s, as a large copy on the same card (5.0; on a card where that copy runs at 4.0, 0.400 ms), but
// not the memory's limit: the single-token linear attention moves equal reads and writes at 5.9 TB/s.  A row's loads,
// reductions and stores follow one another inside its workgroup; non-temporal accesses ran 21% slower.
#pragma once

#include "mma_device.h"

namespace rssm {

struct NormArgs {
  const char* y;
  const char* z;                // or null
  const char* residual;
  const float* post_weight;     // or null
  const float* pre_weight;      // or null
  const float* channel_scale;   // or null
  char* residual_out;
  char* normed;                 // or null
  int64_t y_stride, z_stride, r_stride, ro_stride, n_stride;   // elements
  int32_t rows, C, groups;
  float eps, residual_scale;
};

constexpr int kNormBlock = 256;
constexpr int kNormMaxGroups = 256;

template <int DT>
__device__ __forceinline__ f32x8 load8(const char* p) {
  if constexpr (DT == kF32) {
    const f32x4 a = __builtin_bit_cast(f32x4, ld<false, u32x4>(p)), b = __builtin_bit_cast(f32x4, ld<false, u32x4>(p + 16));
    return stack(a, b);
  } else {
    return from_frag<DT>(__builtin_bit_cast(typename Mma<DT>::frag, ld<false, u32x4>(p)));
  }
}

template <int DT>
__device__ __forceinline__ void store8(char* p, f32x8 v) {
  if constexpr (DT == kF32) {
    st<false>(p, __builtin_bit_cast(u32x4, f32x4{v[0], v[1], v[2], v[3]}));
    st<false>(p + 16, __builtin_bit_cast(u32x4, f32x4{v[4], v[5], v[6], v[7]}));
  } else {
    st<false>(p, __builtin_bit_cast(u32x4, to_frag<DT>(v)));
  }
}

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) v += __shfl_xor(v, d);
  return v;
}

__device__ __forceinline__ float square_sum(f32x8 v) {
  float s = 0.0f;
#pragma unroll
  for (int e = 0; e < 8; ++e) s = fmaf(v[e], v[e], s);
  return s;
}

template <int IT, int RT, int VPT>
__global__ __launch_bounds__(kNormBlock) void block_norm_kernel(NormArgs a) {
  constexpr int ie = sizeof(typename Mma<IT>::elem), re = sizeof(typename Mma<RT>::elem);
  __shared__ float part[2][kNormBlock / 64];
  __shared__ float vec[VPT * kNormBlock];     // grouped norm: one sum a vector of 8 channels
  __shared__ float gsum[kNormMaxGroups];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int nv = a.C / 8;
  const int64_t row = blockIdx.x;
  const char* yp = a.y + row * a.y_stride * ie;
  const char* rp = a.residual + row * a.r_stride * re;
  f32x8 u[VPT], r[VPT];
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int v = tid + i * kNormBlock;
    if (v < nv) {
      u[i] = load8<IT>(yp + v * (8 * ie));
      r[i] = load8<RT>(rp + v * (8 * re));
    } else {
      u[i] = r[i] = f32x8{0, 0, 0, 0, 0, 0, 0, 0};
    }
  }
  if (a.z != nullptr) {
    const char* zp = a.z + row * a.z_stride * ie;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int v = tid + i * kNormBlock;
      if (v < nv) {
        const f32x8 z = load8<IT>(zp + v * (8 * ie));
#pragma unroll
        for (int e = 0; e < 8; ++e) u[i][e] *= silu(z[e]);
      }
    }
  }
  if (a.post_weight != nullptr) {
    const int gv = nv / a.groups;             // vectors a group
    float inv = 0.0f;
    if (a.groups == 1) {
      float s = 0.0f;
#pragma unroll
      for (int i = 0; i < VPT; ++i) s += square_sum(u[i]);
      s = wave_sum(s);
      if (lane == 0) part[0][wave] = s;
      __syncthreads();
      s = (part[0][0] + part[0][1]) + (part[0][2] + part[0][3]);
      inv = 1.0f / sqrtf(s / a.C + a.eps);
    } else {
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        const int v = tid + i * kNormBlock;
        if (v < nv) vec[v] = square_sum(u[i]);
      }
      __syncthreads();
      for (int gi = wave; gi < a.groups; gi += kNormBlock / 64) {
        float s = 0.0f;
        for (int k = lane; k < gv; k += 64) s += vec[gi * gv + k];
        s = wave_sum(s);
        if (lane == 0) gsum[gi] = 1.0f / sqrtf(s / (gv * 8) + a.eps);
      }
      __syncthreads();
    }
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int v = tid + i * kNormBlock;
      if (v < nv) {
        const f32x8 w = load8<kF32>(reinterpret_cast<const char*>(a.post_weight + v * 8));
        u[i] = u[i] * (a.groups == 1 ? inv : gsum[v / gv]) * w;
      }
    }
  }
  float s = 0.0f;
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int v = tid + i * kNormBlock;
    if (v < nv) {
      f32x8 c = u[i] * a.residual_scale;
      if (a.channel_scale != nullptr) c *= load8<kF32>(reinterpret_cast<const char*>(a.channel_scale + v * 8));
      r[i] += c;
      store8<RT>(a.residual_out + row * a.ro_stride * re + v * (8 * re), r[i]);
      s += square_sum(r[i]);
    }
  }
  if (a.normed == nullptr) return;
  s = wave_sum(s);
  if (lane == 0) part[1][wave] = s;
  __syncthreads();
  s = (part[1][0] + part[1][1]) + (part[1][2] + part[1][3]);
  const float inv = 1.0f / sqrtf(s / a.C + a.eps);
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int v = tid + i * kNormBlock;
    if (v < nv) {
      f32x8 n = r[i] * inv;
      if (a.pre_weight != nullptr) n *= load8<kF32>(reinterpret_cast<const char*>(a.pre_weight + v * 8));
      store8<IT>(a.normed + row * a.n_stride * ie + v * (8 * ie), n);
    }
  }
}

}  // namespace rssm
