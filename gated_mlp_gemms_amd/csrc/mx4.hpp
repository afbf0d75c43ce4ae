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

// Eight codes, v[0] in the low half of byte 0, by gfx950's packed conversion: v / scale to the nearest code, ties to the
// even one, saturating (equal to the comparisons of the format's definition for every bf16 value at scales over the whole range).
__device__ __forceinline__ uint32_t mx_codes8(const float (&v)[8], float scale) {
  uint32_t w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(0u, v[0], v[1], scale, 0);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[2], v[3], scale, 1);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[4], v[5], scale, 2);
  return __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[6], v[7], scale, 3);
}

// The value of a code (4 bits): a half of the magnitude's integer, exact.
__device__ __forceinline__ float mx_value(uint32_t c) {
  const uint32_t m = c & 7u, e = m >> 1;
  const float v = e == 0u ? 0.5f * (float)(m & 1u) : __uint_as_float((126u + e) << 23 | (m & 1u) << 22);
  return c & 8u ? -v : v;
}

}  // namespace gmlp
