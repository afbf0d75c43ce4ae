// Kernels of microscaled 4-bit floating point around the products (mx4.h): to blocks along the rows, to blocks of the
// transposed matrix, and back to values. Bound by HBM.
#include "mx4.hpp"
#include "rows.hpp"

namespace gmlp {

namespace {

constexpr int kMxThreads = 256;

// Eight consecutive values of a row as loaded.
template <typename T> struct Oct {
  static constexpr int V = 8 * (int)sizeof(T) / 16;   // 16-byte pieces
  u32x4 p[V];
  __device__ __forceinline__ void load(const void* x, int64_t oct, bool in) {
#pragma unroll
    for (int i = 0; i < V; ++i) p[i] = in ? reinterpret_cast<const u32x4*>(x)[oct * V + i] : u32x4{0u, 0u, 0u, 0u};
  }
  __device__ __forceinline__ void values(float (&v)[8]) const {
    constexpr int N = Piece<T>::N;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      float f[N];
      Piece<T>::unpack(p[i], f);
#pragma unroll
      for (int r = 0; r < N; ++r) v[i * N + r] = f[r];
    }
  }
};

// Blocks along the rows: 8 values a lane, a block four lanes, the scales of 128 values one store.
template <typename T>
__global__ __launch_bounds__(kMxThreads) void mx_rows_kernel(const void* __restrict__ x, int64_t rows, int64_t all,
                                                             int octs, int sh, int64_t plane, int64_t scale_batch,
                                                             uint32_t* __restrict__ codes, uint8_t* __restrict__ scales) {
  const int per = kMxThreads >> sh, lanes = 1 << sh;
  const int wide = (octs + 31) / 32 * 32;   // a plane's octs
  for (int64_t r = (int64_t)blockIdx.x * per + (threadIdx.x >> sh); r < all; r += (int64_t)gridDim.x * per) {
    const int64_t batch = r / rows;
    uint8_t* srow = scales + batch * scale_batch + (r - batch * rows) * 8;
    for (int c = threadIdx.x & (lanes - 1); c < wide; c += lanes) {
      Oct<T> o;
      o.load(x, r * octs + c, c < octs);
      float v[8];
      o.values(v);
      uint32_t top = 0u;
#pragma unroll
      for (int i = 0; i < 8; ++i) top = max(top, __float_as_uint(v[i]) & 0x7fffffffu);
      top = max(top, dpp<0xB1>(top));
      top = max(top, dpp<0x4E>(top));
      const uint32_t s = c < octs ? mx_scale_of(top) : 0u;
      if (c < octs) codes[r * octs + c] = mx_codes8(v, mx_scale_value(s));
      uint32_t four = s << (8 * ((c >> 2) & 3));   // this block's byte among the four of 16 lanes
      four |= dpp<0x124>(four);                    // row_ror:4, row_ror:8
      four |= dpp<0x128>(four);
      if ((c & 15) == 0) *reinterpret_cast<uint32_t*>(srow + (c >> 5) * plane + ((c >> 2) & 4)) = four;
    }
  }
}

// Blocks of the transposed matrix. A wave takes 8 blocks of 32 rows by 8 pieces of 16 bytes of columns, a lane one block of
// one piece's columns: its loads are runs of 128 bytes, and so are its stores of 16 codes' bytes a column, 8 blocks of a
// column being neighbours.
template <typename T>
__global__ __launch_bounds__(64) void mx_columns_kernel(const u32x4* __restrict__ x, int64_t rows, int pieces, int64_t deep,
                                                        int col_tiles, int64_t plane, int64_t scale_batch,
                                                        uint8_t* __restrict__ codes, uint8_t* __restrict__ scales) {
  constexpr int N = Piece<T>::N;   // columns of a piece
  __shared__ uint8_t sc[8 * N][8];
  const int lane = threadIdx.x, o = lane & 7, rb = lane >> 3;
  const int ct = blockIdx.x % col_tiles;
  const int64_t rt = blockIdx.x / col_tiles, batch = blockIdx.y;
  const int c = ct * 8 + o;
  const int64_t cols = (int64_t)pieces * N, r0 = rt * kMxPlane + rb * kMxBlock;
  const bool col = c < pieces;
  const u32x4* src = x + (batch * rows + r0) * pieces + c;
  u32x4 v[kMxBlock];
#pragma unroll
  for (int i = 0; i < kMxBlock; ++i)
    v[i] = col && r0 + i < rows ? src[(int64_t)i * pieces] : u32x4{0u, 0u, 0u, 0u};
  uint8_t* out = codes + (batch * cols + (int64_t)c * N) * (deep / 2) + r0 / 2;
#pragma unroll
  for (int j = 0; j < N; ++j) {
    auto at = [&](int i) -> float {
      if constexpr (N == 4) return __uint_as_float(v[i][j]);
      else return Bits16<T>::to_f32(j & 1 ? v[i][j / 2] >> 16 : v[i][j / 2] & 0xffffu);
    };
    uint32_t top = 0u;
#pragma unroll
    for (int i = 0; i < kMxBlock; ++i) top = max(top, __float_as_uint(at(i)) & 0x7fffffffu);
    const uint32_t s = mx_scale_of(top);
    const float f = mx_scale_value(s);
    u32x4 w;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const float e[8] = {at(8 * q), at(8 * q + 1), at(8 * q + 2), at(8 * q + 3), at(8 * q + 4), at(8 * q + 5), at(8 * q + 6), at(8 * q + 7)};
      w[q] = mx_codes8(e, f);
    }
    if (col && r0 < deep) *reinterpret_cast<u32x4*>(out + (int64_t)j * (deep / 2)) = w;
    sc[o * N + j][rb] = r0 < deep ? (uint8_t)s : 0;
  }
  __syncthreads();
  for (int i = lane; i < 8 * N; i += 64) {
    const int64_t at = (int64_t)ct * 8 * N + i;
    if (at < cols)
      *reinterpret_cast<uint64_t*>(scales + batch * scale_batch + rt * plane + at * 8) = *reinterpret_cast<const uint64_t*>(sc[i]);
  }
}

// Eight values a thread.
template <typename T>
__global__ __launch_bounds__(kMxThreads) void mx_values_kernel(const uint32_t* __restrict__ codes, const uint8_t* __restrict__ scales,
                                                               int64_t rows, int64_t all, int octs, int sh, int64_t plane,
                                                               int64_t scale_batch, u32x4* __restrict__ out) {
  const int per = kMxThreads >> sh, lanes = 1 << sh;
  for (int64_t r = (int64_t)blockIdx.x * per + (threadIdx.x >> sh); r < all; r += (int64_t)gridDim.x * per) {
    const int64_t batch = r / rows;
    const uint8_t* srow = scales + batch * scale_batch + (r - batch * rows) * 8;
    for (int c = threadIdx.x & (lanes - 1); c < octs; c += lanes) {
      const uint32_t w = codes[r * octs + c];
      const float f = mx_scale_value(srow[(c >> 5) * plane + ((c >> 2) & 7)]);
      constexpr int N = Piece<T>::N;
#pragma unroll
      for (int i = 0; i < 8 / N; ++i) {
        float v[N];
#pragma unroll
        for (int k = 0; k < N; ++k) v[k] = mx_value(w >> (4 * (i * N + k))) * f;
        out[(r * octs + c) * (8 / N) + i] = Piece<T>::pack(v);
      }
    }
  }
}

int oct_shift(int octs) {
  int sh = 5;
  while (sh < 8 && (1 << sh) < octs) ++sh;
  return sh;
}

}  // namespace

hipError_t run_mx4_rows(DType dt, const void* x, int64_t batch, int64_t rows, int64_t cols, void* codes, void* scales,
                        hipStream_t s) {
  const int octs = (int)(cols / 8), sh = oct_shift(octs);
  return by_type(dt, [&](auto t) {
    hipLaunchKernelGGL((mx_rows_kernel<decltype(t)>), dim3(item_grid(batch * rows, kMxThreads >> sh)), dim3(kMxThreads), 0, s, x,
                       rows, batch * rows, octs, sh, mx_scale_rows(rows) * 8, mx_scale_bytes(rows, cols),
                       static_cast<uint32_t*>(codes), static_cast<uint8_t*>(scales));
    return hipGetLastError();
  });
}

hipError_t run_mx4_columns(DType dt, const void* x, int64_t batch, int64_t rows, int64_t cols, void* codes, void* scales,
                           hipStream_t s) {
  return by_type(dt, [&](auto t) {
    constexpr int N = Piece<decltype(t)>::N;
    const int pieces = (int)(cols / N), col_tiles = (pieces + 7) / 8;
    const int64_t deep = (rows + kMxBlock - 1) / kMxBlock * kMxBlock;
    hipLaunchKernelGGL((mx_columns_kernel<decltype(t)>), dim3((unsigned)(col_tiles * mx_planes(rows)), (unsigned)batch), dim3(64), 0,
                       s, static_cast<const u32x4*>(x), rows, pieces, deep, col_tiles, mx_scale_rows(cols) * 8,
                       mx_scale_bytes(cols, deep), static_cast<uint8_t*>(codes), static_cast<uint8_t*>(scales));
    return hipGetLastError();
  });
}

hipError_t run_mx4_values(DType dt, const void* codes, const void* scales, int64_t batch, int64_t rows, int64_t K, void* out,
                          hipStream_t s) {
  const int octs = (int)(K / 8), sh = oct_shift(octs);
  return by_type(dt, [&](auto t) {
    hipLaunchKernelGGL((mx_values_kernel<decltype(t)>), dim3(item_grid(batch * rows, kMxThreads >> sh)), dim3(kMxThreads), 0, s,
                       static_cast<const uint32_t*>(codes), static_cast<const uint8_t*>(scales), rows, batch * rows, octs, sh,
                       mx_scale_rows(rows) * 8, mx_scale_bytes(rows, K), static_cast<u32x4*>(out));
    return hipGetLastError();
  });
}

}  // namespace gmlp
