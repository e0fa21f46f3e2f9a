// Row operators' shared pieces: 8 consecutive elements of a row as fp32,
// reductions over the lanes of a block of 128 columns and over a row, and the
// 8-bit formats with their block scales.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/tss.h"
#include "gemm_kernel.h"
#include "groups.h"

namespace tss {

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

constexpr int kScaleBlock = 128;          // columns that share a scale
constexpr float kSmallestAmax = 1e-30f;   // a block's largest magnitude is taken as at least this (its scale stays
                                          // a normal number with a finite reciprocal)

struct E4M3 {};
struct E5M2 {};
struct I8 {};  // -127 .. 127
template <typename Q>
constexpr float kLargest = __is_same(Q, E4M3) ? 448.0f : __is_same(Q, I8) ? 127.0f : 57344.0f;

// 8 consecutive elements as they are in memory: 16 bytes (fp16, bf16) or 32
// (fp32), loaded with 16-byte accesses and widened when they are used.
template <typename T>
struct Raw8 {
  u32x4 v[sizeof(T) / 2];
};

template <typename T>
__device__ __forceinline__ Raw8<T> load8(const T *p) {
  Raw8<T> r;
#pragma unroll
  for (int i = 0; i < int(sizeof(T) / 2); ++i) r.v[i] = reinterpret_cast<const u32x4 *>(p)[i];
  return r;
}

template <typename T>
__device__ __forceinline__ Raw8<T> zero8() {
  Raw8<T> r;
#pragma unroll
  for (int i = 0; i < int(sizeof(T) / 2); ++i) r.v[i] = u32x4{0, 0, 0, 0};
  return r;
}

template <typename T>
__device__ __forceinline__ void widen8(const Raw8<T> &r, float (&f)[8]) {
  if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t w = r.v[i / 4][i % 4];  // a value: bit_cast of a vector's element by reference reads its first
      f[i] = __builtin_bit_cast(float, w);
    }
  } else if constexpr (__is_same(T, __bf16)) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = __builtin_bit_cast(float, r.v[0][i] << 16);
      f[2 * i + 1] = __builtin_bit_cast(float, r.v[0][i] & 0xffff0000u);
    }
  } else {
    const f16x8 h = __builtin_bit_cast(f16x8, r.v[0]);
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = float(h[i]);
  }
}

// Rounded to nearest even.
template <typename T>
__device__ __forceinline__ void store8(T *p, const float (&f)[8]) {
  if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int i = 0; i < 2; ++i)
      reinterpret_cast<f32x4 *>(p)[i] = f32x4{f[4 * i], f[4 * i + 1], f[4 * i + 2], f[4 * i + 3]};
  } else {
    typedef T T8 __attribute__((ext_vector_type(8)));
    T8 h;
#pragma unroll
    for (int i = 0; i < 8; ++i) h[i] = (T)f[i];
    *reinterpret_cast<T8 *>(p) = h;
  }
}

// The same past the caches, for outputs that they would not hold anyway.
template <typename T>
__device__ __forceinline__ void store8_streamed(T *p, const float (&f)[8]) {
  if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int i = 0; i < 2; ++i)
      __builtin_nontemporal_store(f32x4{f[4 * i], f[4 * i + 1], f[4 * i + 2], f[4 * i + 3]}, reinterpret_cast<f32x4 *>(p) + i);
  } else {
    typedef T T8 __attribute__((ext_vector_type(8)));
    T8 h;
#pragma unroll
    for (int i = 0; i < 8; ++i) h[i] = (T)f[i];
    __builtin_nontemporal_store(h, reinterpret_cast<T8 *>(p));
  }
}

// |a|, |b| to the larger, NaN if either is NaN.
__device__ __forceinline__ float max_abs(float a, float b) {
  return __builtin_elementwise_maximum(__builtin_fabsf(a), __builtin_fabsf(b));
}

// Rotation by N lanes within each 16 lanes.
template <int N>
__device__ __forceinline__ float rot16(float v) {
  return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), 0x120 + N, 0xf, 0xf, false));
}

// Over the 16 lanes that hold one block of 128 columns (8 each); every lane gets the result.
__device__ __forceinline__ float max16(float v) {
  v = __builtin_elementwise_maximum(v, rot16<8>(v));
  v = __builtin_elementwise_maximum(v, rot16<4>(v));
  v = __builtin_elementwise_maximum(v, rot16<2>(v));
  return __builtin_elementwise_maximum(v, rot16<1>(v));
}

__device__ __forceinline__ float min16(float v) {
  v = fminf(v, rot16<8>(v));
  v = fminf(v, rot16<4>(v));
  v = fminf(v, rot16<2>(v));
  return fminf(v, rot16<1>(v));
}

__device__ __forceinline__ float sum64(float v) {
  v += rot16<8>(v);
  v += rot16<4>(v);
  v += rot16<2>(v);
  v += rot16<1>(v);
  v += __shfl_xor(v, 16);
  return v + __shfl_xor(v, 32);
}

// Sum (largest magnitude) over L neighbouring lanes, L a power of two; every
// lane gets the same bits.
template <int CTRL>
__device__ __forceinline__ float lane_swap(float v) {
  return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), CTRL, 0xf, 0xf, false));
}
template <int L, typename F>
__device__ __forceinline__ float over_lanes(float v, F join) {
  if constexpr (L >= 2) v = join(v, lane_swap<0xb1>(v));    // lanes 1 0 3 2 of four
  if constexpr (L >= 4) v = join(v, lane_swap<0x4e>(v));    // 2 3 0 1
  if constexpr (L >= 8) v = join(v, lane_swap<0x141>(v));   // eight mirrored
  if constexpr (L >= 16) v = join(v, lane_swap<0x140>(v));  // sixteen mirrored
  if constexpr (L >= 32) v = join(v, __shfl_xor(v, 16));
  if constexpr (L >= 64) v = join(v, __shfl_xor(v, 32));
  return v;
}
template <int L>
__device__ __forceinline__ float sum_lanes(float v) {
  return over_lanes<L>(v, [](float a, float b) { return a + b; });
}
template <int L>
__device__ __forceinline__ float max_lanes(float v) {
  return over_lanes<L>(v, [](float a, float b) { return __builtin_elementwise_maximum(a, b); });
}

// A block's scale = amax / largest value of the type, and what v / scale takes:
// the quotient is the product with the reciprocal, corrected once by its
// remainder, which rounds it as a division does for 2 more operations an
// element (the bare product moves some of the values that lie on a rounding
// border of the 8-bit type, as many of those of a 16-bit type do).  |v| <= amax keeps the
// quotient below the halfway point past the largest value, so the conversion
// needs no clamp.  Integers have few values, and halves between them are
// common quotients (x = amax / 2 is 63.5), so theirs is the quotient by amax /
// 127 itself, not by its rounding to fp32: `low` is what the rounding left out.
template <typename Q>
struct BlockScale {
  float scale, inv, back, low;
  explicit __device__ __forceinline__ BlockScale(float amax) {
    scale = __builtin_elementwise_maximum(amax, kSmallestAmax) / kLargest<Q>;
    const float r = __builtin_amdgcn_rcpf(scale);
    // an infinite scale: finite values are 0, infinite ones NaN; integers, which have no NaN: also of a NaN scale
    const bool inf = __is_same(Q, I8) ? !(scale < __builtin_inff()) : scale == __builtin_inff();
    inv = inf ? 0.0f : __builtin_fmaf(__builtin_fmaf(-scale, r, 1.0f), r, r);
    back = inf ? 0.0f : -scale;
    low = inf ? 0.0f : __builtin_fmaf(-kLargest<Q>, scale, __builtin_elementwise_maximum(amax, kSmallestAmax)) / -kLargest<Q>;
  }
  __device__ __forceinline__ float quotient(float v) const {
    const float t = v * inv;
    if constexpr (__is_same(Q, I8)) return __builtin_fmaf(__builtin_fmaf(t, low, __builtin_fmaf(t, back, v)), inv, t);
    return __builtin_fmaf(__builtin_fmaf(t, back, v), inv, t);
  }
};

// 8 quotients, rounded to the type.
template <typename Q>
__device__ __forceinline__ u32x2 round8(const float (&f)[8]) {
  u32x2 r;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    int w = 0;
    if constexpr (__is_same(Q, I8)) {
      // 1.5 * 2^23 added: the sum's last byte is the rounded quotient in two's complement; 0 of a NaN
      uint32_t b[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float q = f[4 * i + j];
        b[j] = __builtin_bit_cast(uint32_t, (q == q ? q : 0.0f) + 0x1.8p23f);
      }
      const uint32_t lo = __builtin_amdgcn_perm(b[1], b[0], 0x0c0c0400u), hi = __builtin_amdgcn_perm(b[3], b[2], 0x04000c0cu);
      w = int(lo | hi);
    } else if constexpr (__is_same(Q, E4M3)) {
      w = __builtin_amdgcn_cvt_pk_fp8_f32(f[4 * i], f[4 * i + 1], w, false);
      w = __builtin_amdgcn_cvt_pk_fp8_f32(f[4 * i + 2], f[4 * i + 3], w, true);
    } else {
      w = __builtin_amdgcn_cvt_pk_bf8_f32(f[4 * i], f[4 * i + 1], w, false);
      w = __builtin_amdgcn_cvt_pk_bf8_f32(f[4 * i + 2], f[4 * i + 3], w, true);
    }
    r[i] = uint32_t(w);
  }
  return r;
}

template <typename Q>
__device__ __forceinline__ u32x2 pack8(const float (&v)[8], const BlockScale<Q> &s) {
  float f[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) f[i] = s.quotient(v[i]);
  return round8<Q>(f);
}

}  // namespace tss
