// mma_device.h -- matrix-core fragments shared by the prompt-side kernels
// (linear attention, paged attention) on gfx950.
//
// One product step is D[16][16] += A[16][32] Bm[32][16].  Operand fragments hold 8
// elements a lane: lane l has row (A) or column (Bm) l % 16 and the eight
// contraction indexes of its lane group g = l / 16.  D has 4 rows a lane: column l % 16,
// rows 4g .. 4g + 3.  The 16-bit types use one 16x16x32 instruction; fp32
// takes eight 16x16x4 ones, step e consuming element e of every lane, so both
// see the same fragment.  The order of the contraction indexes is free as long as
// A and Bm agree, and two orders are used:
//   straight   element e of group g is index 8g + e (16 contiguous bytes of a
//              row-major tile with the contraction along the row);
//   split      element e < 4 is 4g + e, e >= 4 is 16 + 4g + (e - 4): the
//              rows that group g holds of two stacked D tiles.  A product's
//              D tiles become the next product's operand without leaving the
//              registers, and the other operand comes by columns of a
//              row-major tile (the transposing LDS read for 16-bit types).
#pragma once

#include "rssm_device.h"

namespace rssm {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef short i16x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x8 __attribute__((ext_vector_type(8)));

template <int IT> struct Mma;
template <> struct Mma<kBF16> {
  typedef uint16_t elem;       // storage in LDS and global memory
  typedef bf16x8 frag;
};
template <> struct Mma<kF16> {
  typedef uint16_t elem;
  typedef f16x8 frag;
};
template <> struct Mma<kF32> {
  typedef float elem;
  typedef f32x8 frag;
};

template <int IT>
__device__ __forceinline__ f32x4 mma(typename Mma<IT>::frag a, typename Mma<IT>::frag b, f32x4 c) {
  if constexpr (IT == kBF16) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
  } else if constexpr (IT == kF16) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a[e], b[e], c, 0, 0, 0);
    return c;
  }
}

// Eight fp32 values rounded once (nearest even) to the operand type.
template <int IT>
__device__ __forceinline__ typename Mma<IT>::frag to_frag(f32x8 v) {
  return __builtin_convertvector(v, typename Mma<IT>::frag);
}

// The leading 8 significant bits of each value as bf16 (cut off, so that three turns
// take all 24 exactly); `v` keeps the rest.
__device__ __forceinline__ bf16x8 take_bf16(f32x8& v) {
  u32x4 p;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t a = __float_as_uint(v[2 * i]), b = __float_as_uint(v[2 * i + 1]);
    p[i] = __builtin_amdgcn_perm(b, a, 0x07060302u);
    v[2 * i] -= __uint_as_float(a & 0xffff0000u);
    v[2 * i + 1] -= __uint_as_float(b & 0xffff0000u);
  }
  return __builtin_bit_cast(bf16x8, p);
}

template <int IT>
__device__ __forceinline__ f32x8 from_frag(typename Mma<IT>::frag v) {
  return __builtin_convertvector(v, f32x8);
}

// Straight fragment: 8 contiguous elements at p (16-byte aligned).
template <int IT>
__device__ __forceinline__ typename Mma<IT>::frag frag_row(const typename Mma<IT>::elem* p) {
  if constexpr (IT == kF32) {
    const f32x4 a = *reinterpret_cast<const f32x4*>(p), b = *reinterpret_cast<const f32x4*>(p + 4);
    return f32x8{a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
  } else {
    return __builtin_bit_cast(typename Mma<IT>::frag, *reinterpret_cast<const u32x4*>(p));
  }
}

// Row pitch, in elements, of an LDS tile of `cols` (64 or 128) columns.  16-bit: rows
// start 8 banks apart (an odd multiple of 32 bytes), so that the 4 rows x 32 bytes of a
// transposing read and the 8 rows x 16 bytes of a straight one fall on different banks.
// fp32: 4 banks apart.
template <int IT>
constexpr int tile_pitch(int cols) {
  return IT == kF32 ? cols + 4 : cols + 16;
}

// Split fragment by columns of a row-major LDS tile: lane l takes column
// c0 + l % 16 of rows r0 + {4g .. 4g+3} and r0 + 16 + {4g .. 4g+3}.  16-bit: the
// transposing read hands each lane of a 16-lane group one column of the 4x16 block
// whose row q, columns 4k .. 4k+3 lane 4q + k addresses.
// kStep: distance between the lanes' groups of 4 columns (4: consecutive columns).
template <int IT, int kStep = 4>
__device__ __forceinline__ typename Mma<IT>::frag frag_col(const typename Mma<IT>::elem* tile, int stride, int r0,
                                                           int c0, int lane) {
  const int g = lane >> 4, i = lane & 15;
  if constexpr (IT == kF32) {
    const float* p = tile + (r0 + 4 * g) * stride + c0 + kStep * (i >> 2) + (i & 3);
    f32x8 v;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      v[e] = p[e * stride];
      v[e + 4] = p[(16 + e) * stride];
    }
    return v;
  } else {
    typedef __attribute__((address_space(3))) i16x4 lds_i16x4;
    const uint16_t* p = tile + (r0 + 4 * g + (i >> 2)) * stride + c0 + (i & 3) * kStep;
    const i16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4*)(p));
    const i16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4*)(p + 16 * stride));
    const u32x2 a = __builtin_bit_cast(u32x2, lo), b = __builtin_bit_cast(u32x2, hi);
    return __builtin_bit_cast(typename Mma<IT>::frag, u32x4{a.x, a.y, b.x, b.y});
  }
}

// c plus the infinities and NaN of x that a lane's column sees, those whose weight
// p is not zero (a product would make 0 times infinity a NaN).  Products of 0s and 1s count
// the +infinities and -infinities among the terms (a NaN counts as both).
template <int IT>
__device__ __forceinline__ f32x4 add_odd(f32x8 x, typename Mma<IT>::frag p, f32x4 c) {
  __builtin_amdgcn_sched_barrier(0);   // rare: one call's registers at a time
  const f32x8 w = from_frag<IT>(p);
  f32x8 pos, neg, plus, minus;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const bool odd = !(fabsf(x[e]) < __builtin_inff());
    pos[e] = odd && x[e] != -__builtin_inff() ? 1.0f : 0.0f;
    neg[e] = odd && x[e] != __builtin_inff() ? 1.0f : 0.0f;
    plus[e] = w[e] >= 0.0f ? (w[e] > 0.0f ? 1.0f : 0.0f) : (w[e] < 0.0f ? 0.0f : 1.0f);
    minus[e] = w[e] <= 0.0f ? (w[e] < 0.0f ? 1.0f : 0.0f) : (w[e] > 0.0f ? 0.0f : 1.0f);
  }
  typedef typename Mma<IT>::frag frag;
  const f32x4 zero = f32x4{0, 0, 0, 0};
  const frag fp = to_frag<IT>(pos), fn = to_frag<IT>(neg), sp = to_frag<IT>(plus), sm = to_frag<IT>(minus);
  const f32x4 up = mma<IT>(fn, sm, mma<IT>(fp, sp, zero)), down = mma<IT>(fp, sm, mma<IT>(fn, sp, zero));
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    if (up[r] != 0.0f) c[r] += __builtin_inff();
    if (down[r] != 0.0f) c[r] -= __builtin_inff();
  }
  return c;
}

// x with zeros for infinities and NaN.
template <int IT>
__device__ __forceinline__ typename Mma<IT>::frag finite_part(f32x8 x) {
#pragma unroll
  for (int e = 0; e < 8; ++e) x[e] = fabsf(x[e]) < __builtin_inff() ? x[e] : 0.0f;
  return to_frag<IT>(x);
}

// c + x p where x may hold infinities and NaN: the finite part by a product, the rest by add_odd.
template <int IT>
__device__ __forceinline__ f32x4 mma_seen(typename Mma<IT>::frag v, typename Mma<IT>::frag p, f32x4 c) {
  const f32x8 x = from_frag<IT>(v);
  return add_odd<IT>(x, p, mma<IT>(finite_part<IT>(x), p, c));
}

// Split fragment of two stacked D tiles.
__device__ __forceinline__ f32x8 stack(f32x4 a, f32x4 b) {
  return f32x8{a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
}

// One element in storage, widened.
template <int IT>
__device__ __forceinline__ float elem_to_float(typename Mma<IT>::elem v) {
  if constexpr (IT == kF32) return v;
  else if constexpr (IT == kBF16) return __uint_as_float(static_cast<uint32_t>(v) << 16);
  else return f16_bits_to_float(v);
}

// Four consecutive elements in storage <-> fp32.
template <int IT>
__device__ __forceinline__ f32x4 widen4(const typename Mma<IT>::elem* p) {
  if constexpr (IT == kF32) {
    return *reinterpret_cast<const f32x4*>(p);
  } else {
    const u32x2 w = *reinterpret_cast<const u32x2*>(p);
    if constexpr (IT == kBF16) {
      return f32x4{__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xffff0000u), __uint_as_float(w.y << 16),
                   __uint_as_float(w.y & 0xffff0000u)};
    } else {
      return f32x4{f16_bits_to_float(w.x & 0xffffu), f16_bits_to_float(w.x >> 16), f16_bits_to_float(w.y & 0xffffu),
                   f16_bits_to_float(w.y >> 16)};
    }
  }
}

typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
typedef _Float16 f16x4 __attribute__((ext_vector_type(4)));

template <int IT>
__device__ __forceinline__ void narrow4(typename Mma<IT>::elem* p, f32x4 v) {
  if constexpr (IT == kF32) {
    *reinterpret_cast<f32x4*>(p) = v;
  } else if constexpr (IT == kBF16) {
    *reinterpret_cast<u32x2*>(p) = __builtin_bit_cast(u32x2, __builtin_convertvector(v, bf16x4));
  } else {
    *reinterpret_cast<u32x2*>(p) = __builtin_bit_cast(u32x2, __builtin_convertvector(v, f16x4));
  }
}

// Eight consecutive elements in global memory <-> fp32 (16-byte aligned; rounded once).
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

// Largest value, and sum, over the four lane groups that share a column.
__device__ __forceinline__ float max_groups(float v) {
  v = fmaxf(v, __shfl_xor(v, 16));
  return fmaxf(v, __shfl_xor(v, 32));
}
__device__ __forceinline__ float sum_groups(float v) {
  v += __shfl_xor(v, 16);
  return v + __shfl_xor(v, 32);
}

// v / (1 + exp(-v)) by the hardware's exp2 and reciprocal (each within one unit
// of the last place; the argument's rounding adds 2^-24 |v|, which only matters where
// the result is tiny).  exp overflows to infinity for very negative v: the result is -0.
__device__ __forceinline__ float silu(float v) {
  return v * __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(v * -1.4426950408889634f));
}

// Workgroup order that gives each of the 8 XCDs (workgroups are dealt to them in
// turn) one contiguous range of items, so that neighbouring items, which
// share inputs, meet in one L2.
__device__ __forceinline__ int xcd_order(int block, int total) {
  constexpr int kXcds = 8;
  const int per = total / kXcds, extra = total % kXcds;
  const int x = block % kXcds, i = block / kXcds;
  return x * per + (x < extra ? x : extra) + i;
}

}  // namespace rssm
