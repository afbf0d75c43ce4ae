// What the kernels that go over rows share: single elements and 16-byte pieces of the three element types,
// reductions over the lanes of a row, launch sizes.
#pragma once

#include <algorithm>

#include "common.hpp"
#include "launch.hpp"

namespace gmlp {

template <typename T> __device__ __forceinline__ float load1(const void* p, int64_t i) {
  if constexpr (sizeof(T) == 4) return reinterpret_cast<const float*>(p)[i];
  else return Bits16<T>::to_f32(reinterpret_cast<const uint16_t*>(p)[i]);
}
template <typename T> __device__ __forceinline__ void store1(void* p, int64_t i, float v) {
  if constexpr (sizeof(T) == 4) reinterpret_cast<float*>(p)[i] = v;
  else reinterpret_cast<uint16_t*>(p)[i] = (uint16_t)Bits16<T>::from_f32(v);
}

// ---- reductions over the L lanes of a token (a power of two, 16 .. 64), result in every lane --
// Inside 16 lanes the partner is reached by a DPP operand (quad permutes, then the mirrors of 8 and
// 16 lanes, which after the quad steps pair the same halves as xor 4 and xor 8 would).

template <int CTRL> __device__ __forceinline__ uint32_t dpp(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp((int)v, (int)v, CTRL, 0xf, 0xf, false);
}
template <int L, typename Op> __device__ __forceinline__ uint32_t group_reduce(uint32_t v, Op op) {
  v = op(v, dpp<0xB1>(v));    // lanes 1 0 3 2
  v = op(v, dpp<0x4E>(v));    // lanes 2 3 0 1
  v = op(v, dpp<0x141>(v));   // mirror of 8
  v = op(v, dpp<0x140>(v));   // mirror of 16
#pragma unroll
  for (int o = 16; o < L; o <<= 1) v = op(v, (uint32_t)__shfl_xor((int)v, o));
  return v;
}
template <int L> __device__ __forceinline__ uint32_t group_max(uint32_t v) {
  return group_reduce<L>(v, [](uint32_t a, uint32_t b) { return max(a, b); });
}
template <int L> __device__ __forceinline__ uint32_t group_min(uint32_t v) {
  return group_reduce<L>(v, [](uint32_t a, uint32_t b) { return min(a, b); });
}
template <int L> __device__ __forceinline__ float group_sum(float v) {
  return __uint_as_float(group_reduce<L>(__float_as_uint(v), [](uint32_t a, uint32_t b) {
    return __float_as_uint(__uint_as_float(a) + __uint_as_float(b));
  }));
}

template <typename T> struct Piece {   // 16 bytes of a row
  static constexpr int N = 16 / (int)sizeof(T);
  static __device__ __forceinline__ void unpack(const u32x4 x, float (&v)[N]) {
    if constexpr (N == 4) {
#pragma unroll
      for (int r = 0; r < 4; ++r) v[r] = __uint_as_float(x[r]);
    } else {
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        v[2 * r] = Bits16<T>::to_f32(x[r] & 0xffffu);
        v[2 * r + 1] = Bits16<T>::to_f32(x[r] >> 16);
      }
    }
  }
  static __device__ __forceinline__ u32x4 pack(const float (&v)[N]) {
    if constexpr (N == 4)
      return u32x4{__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3])};
    else
      return u32x4{pack16x2<T>(v[0], v[1]), pack16x2<T>(v[2], v[3]), pack16x2<T>(v[4], v[5]), pack16x2<T>(v[6], v[7])};
  }
};

template <bool NT> __device__ __forceinline__ u32x4 load_piece(const u32x4* p) {
  if constexpr (NT) return __builtin_nontemporal_load(p);
  else return *p;
}
template <bool NT> __device__ __forceinline__ void store_piece(u32x4* p, u32x4 v) {
  if constexpr (NT) __builtin_nontemporal_store(v, p);
  else *p = v;
}

// Workgroups for `items` items, `per` a workgroup: at most 2^20, which then take several (2^32 threads are more
// than a launch can have).
inline unsigned item_grid(int64_t items, int64_t per) { return (unsigned)std::min<int64_t>((items + per - 1) / per, 1 << 20); }

// f() with the element type of `dt` as its argument.
template <typename F> hipError_t by_type(DType dt, F f) {
  switch (dt) {
    case DT_F32: return f(float{});
    case DT_BF16: return f(bf16{});
    case DT_F16: return f(f16{});
    default: return hipErrorInvalidValue;
  }
}

}  // namespace gmlp
