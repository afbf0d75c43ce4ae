// Device and host pieces of microscaled 4-bit floating point (mx4.h) that its kernels share.
#pragma once

#include <stdint.h>

#include "common.hpp"

namespace gmlp {

constexpr int kMxBlock = 32;       // values that share a scale
constexpr int kMxPlane = 256;      // values of a row whose scales are together
inline int64_t mx_planes(int64_t K) { return (K + kMxPlane - 1) / kMxPlane; }
inline int64_t mx_scale_rows(int64_t rows) { return (rows / 4 + 1) * 4; }
inline int64_t mx_scale_bytes(int64_t rows, int64_t K) { return mx_planes(K) * mx_scale_rows(rows) * 8; }

// The scale byte of a block whose largest magnitude has the fp32 bits `top` (an infinity or a NaN: above every number):
// the exponent less e2m1's own largest (6 = 1.5 x 2^2). fp32 subnormals have exponent 0, as 2^-127's byte.
__device__ __forceinline__ uint32_t mx_scale_of(uint32_t top) {
  const uint32_t e = top >> 23;
  return e == 255u ? 255u : e > 2u ? e - 2u : 0u;
}
// What the conversions and a value are divided or multiplied by; 2^-127 is subnormal.
__device__ __forceinline__ float mx_scale_value(uint32_t s) {
  return s == 255u ? __builtin_nanf("") : __uint_as_float(s == 0u ? 0x00400000u : s << 23);
}

// Of 16-bit pairs: the larger magnitudes by halves, the larger half.
typedef unsigned short u16x2 __attribute__((ext_vector_type(2)));
__device__ __forceinline__ uint32_t mx_max16(uint32_t a, uint32_t b) {
  return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(u16x2, a & 0x7fff7fffu),
                                                                __builtin_bit_cast(u16x2, b & 0x7fff7fffu)));
}
__device__ __forceinline__ uint32_t mx_top16(uint32_t m) { return max(m >> 16, m & 0xffffu); }
// The fp32 bits of a value of T's bits.
template <typename T> __device__ __forceinline__ uint32_t mx_f32_bits(uint32_t v) {
  if constexpr (sizeof(T) == 4) return v;
  else return __float_as_uint(Bits16<T>::to_f32(v));
}

// Eight codes, the first value's in the low half of byte 0, by gfx950's packed conversions: v / scale to the nearest code, ties to the
// even one, saturating (equal to the comparisons of the format's definition for every 16-bit value at scales over the whole range).
__device__ __forceinline__ uint32_t mx_codes8(const u32x4& a, const u32x4& b, float scale) {
  uint32_t w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(0u, __uint_as_float(a[0]), __uint_as_float(a[1]), scale, 0);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, __uint_as_float(a[2]), __uint_as_float(a[3]), scale, 1);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, __uint_as_float(b[0]), __uint_as_float(b[1]), scale, 2);
  return __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, __uint_as_float(b[2]), __uint_as_float(b[3]), scale, 3);
}
template <typename T, int S> __device__ __forceinline__ uint32_t mx_codes2(uint32_t w, uint32_t pair, float scale) {
  typedef T T2 __attribute__((ext_vector_type(2)));
  if constexpr (std::is_same<T, _Float16>::value)
    return __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(w, __builtin_bit_cast(T2, pair), scale, S);
  else
    return __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(w, __builtin_bit_cast(T2, pair), scale, S);
}
template <typename T> __device__ __forceinline__ uint32_t mx_codes8(uint32_t a, uint32_t b, uint32_t c, uint32_t d, float scale) {
  return mx_codes2<T, 3>(mx_codes2<T, 2>(mx_codes2<T, 1>(mx_codes2<T, 0>(0u, a, scale), b, scale), c, scale), d, scale);
}

// The values of eight codes times the scale, rounded to T (exact but for T's subnormals and infinities).
template <typename T, int S> __device__ __forceinline__ uint32_t mx_values2(uint32_t w, float scale) {
  if constexpr (std::is_same<T, _Float16>::value)
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, scale, S));
  else
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, S));
}
template <typename T> __device__ __forceinline__ void mx_values8(uint32_t w, float scale, u32x4 (&v)[sizeof(T) / 2]) {
  if constexpr (sizeof(T) == 2) {
    v[0] = u32x4{mx_values2<T, 0>(w, scale), mx_values2<T, 1>(w, scale), mx_values2<T, 2>(w, scale), mx_values2<T, 3>(w, scale)};
  } else {
    auto two = [](auto f, u32x4& to, int at) {
      to[at] = __float_as_uint(f[0]);
      to[at + 1] = __float_as_uint(f[1]);
    };
    two(__builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, scale, 0), v[0], 0);
    two(__builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, scale, 1), v[0], 2);
    two(__builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, scale, 2), v[1], 0);
    two(__builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, scale, 3), v[1], 2);
  }
}

}  // namespace gmlp
