// Kernels of microscaled 4-bit floating point around the products (mx4.h): to blocks along the rows, to blocks of the
// transposed matrix, and back to values. Bound by HBM.
#include "mx4.hpp"
#include "rows.hpp"

namespace gmlp {

namespace {

constexpr int kMxThreads = 256;
template <typename T> constexpr int kMxLoads = sizeof(T) == 4 ? 2 : 4;   // rows of a half wave

// A lane's eight values of a row in 16-byte pieces, their largest magnitude as T's own bits (those of magnitudes are in the
// values' order, infinities and NaNs above), and their codes. 16-bit pairs are converted as they are, without fp32 between.
template <typename T> struct Oct {
  static constexpr int V = 8 * (int)sizeof(T) / 16;
  u32x4 p[V];
  __device__ __forceinline__ void load(const u32x4* x, bool in) {
#pragma unroll
    for (int i = 0; i < V; ++i) p[i] = in ? x[i] : u32x4{0u, 0u, 0u, 0u};
  }
  __device__ __forceinline__ uint32_t top() const {
    if constexpr (V == 1) {
      return mx_top16(mx_max16(mx_max16(p[0][0], p[0][1]), mx_max16(p[0][2], p[0][3])));
    } else {
      uint32_t t = 0u;
#pragma unroll
      for (int i = 0; i < 8; ++i) t = max(t, p[i / 4][i % 4] & 0x7fffffffu);
      return t;
    }
  }
  __device__ __forceinline__ uint32_t codes(float scale) const {
    if constexpr (V == 1) return mx_codes8<T>(p[0][0], p[0][1], p[0][2], p[0][3], scale);
    else return mx_codes8(p[0], p[1], scale);
  }
};

// Blocks along the rows: 8 values a lane and a block four lanes, so a row's 256 values with a plane of scales are a half wave's,
// and a wave's U loads, made before the first is used, are U pairs of rows (8192 x 4096 of bf16, us, a row after the other at
// 16 bytes a lane 21; U 2 / 4 / 8 / 16: 16.2, 15.5, 17.1, 20.5).
template <typename T>
__global__ __launch_bounds__(kMxThreads) void mx_rows_kernel(const u32x4* __restrict__ x, int64_t rows, int octs, int planes,
                                                             int64_t units, int64_t plane, int64_t scale_batch,
                                                             uint32_t* __restrict__ codes, uint8_t* __restrict__ scales) {
  constexpr int U = kMxLoads<T>, V = Oct<T>::V;
  const int lane = threadIdx.x & 63, o = lane & 31, half = lane >> 5;
  const int64_t batch = blockIdx.y;
  x += batch * rows * octs * V;
  codes += batch * rows * octs;
  scales += batch * scale_batch;
  for (int64_t unit = (int64_t)blockIdx.x * (kMxThreads / 64) + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6); unit < units;
       unit += (int64_t)gridDim.x * (kMxThreads / 64)) {
    const int64_t rt = unit / planes, r0 = rt * 2 * U + half;
    const int at = (int)(unit - rt * planes), c = at * 32 + o;
    const bool in = c < octs;
    Oct<T> v[U];
#pragma unroll
    for (int i = 0; i < U; ++i) v[i].load(x + ((r0 + 2 * i) * octs + c) * V, in && r0 + 2 * i < rows);
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int64_t r = r0 + 2 * i;
      uint32_t top = v[i].top();
      top = max(top, dpp<0xB1>(top));
      top = max(top, dpp<0x4E>(top));
      const uint32_t s = mx_scale_of(mx_f32_bits<T>(top));   // (0 behind the row's last block)
      const uint32_t w = v[i].codes(mx_scale_value(s));
      uint32_t four = s << (8 * ((o >> 2) & 3));   // this block's byte among the four of 16 lanes
      four |= dpp<0x124>(four);                    // row_ror:4, row_ror:8
      four |= dpp<0x128>(four);
      if (r < rows) {
        if (in) codes[r * octs + c] = w;
        if ((o & 15) == 0) *reinterpret_cast<uint32_t*>(scales + at * plane + r * 8 + (o >> 2)) = four;
      }
    }
  }
}

// Blocks of the transposed matrix, and with ROWS (16-bit types) those along its rows from the same registers. A wave takes 8 blocks
// of 32 rows by 8 pieces of 16 bytes of columns, a lane one block of one piece's columns: its loads are runs of 128
// bytes, and so are its stores of 16 codes' bytes a column, 8 blocks of a column being neighbours. For the rows four lanes
// next to one another hold a block, and W = 4 waves a whole plane of columns (8192 x 4096 of bf16, us: two launches 32.5, one
// 29.5 and, held to the registers of two waves a SIMD, 23.5).
template <typename T, int W, bool ROWS>
__global__ __launch_bounds__(64 * W) __attribute__((amdgpu_waves_per_eu(ROWS ? 2 : 3))) void mx_columns_kernel(const u32x4* __restrict__ x, int64_t rows, int pieces, int64_t deep,
                                                            int col_tiles, int64_t plane, int64_t scale_batch,
                                                            uint8_t* __restrict__ codes, uint8_t* __restrict__ scales,
                                                            int64_t row_plane, int64_t row_batch,
                                                            uint32_t* __restrict__ row_codes, uint8_t* __restrict__ row_scales) {
  constexpr int N = Piece<T>::N, C = 8 * N * W;   // columns of a piece, of a workgroup
  static_assert(!ROWS || (N == 8 && C == kMxPlane), "rows need a plane of 16-bit columns");
  __shared__ __attribute__((aligned(16))) uint8_t sc[C][8];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, o = lane & 7, rb = lane >> 3;
  const int ct = blockIdx.x % col_tiles;
  const int64_t rt = blockIdx.x / col_tiles, batch = blockIdx.y;
  const int c = (ct * W + wave) * 8 + o;
  const int64_t cols = (int64_t)pieces * N, r0 = rt * kMxPlane + rb * kMxBlock;
  const bool col = c < pieces;
  const u32x4* src = x + (batch * rows + r0) * pieces + c;
  u32x4 v[kMxBlock];
#pragma unroll
  for (int i = 0; i < kMxBlock; ++i)
    v[i] = col && r0 + i < rows ? src[(int64_t)i * pieces] : u32x4{0u, 0u, 0u, 0u};
  if constexpr (ROWS) {
    __shared__ uint32_t rs[8][kMxPlane / 4];   // the scales of the plane's 8 blocks, of four rows a word
    uint32_t* out = row_codes + (batch * rows + r0) * pieces + c;
#pragma unroll
    for (int i = 0; i < kMxBlock; i += 4) {
      uint32_t four = 0u;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const u32x4 q = v[i + k];
        uint32_t top = mx_top16(mx_max16(mx_max16(q[0], q[1]), mx_max16(q[2], q[3])));
        top = max(top, dpp<0xB1>(top));
        top = max(top, dpp<0x4E>(top));
        const uint32_t s = mx_scale_of(mx_f32_bits<T>(top));
        if (col && r0 + i + k < rows) out[(int64_t)(i + k) * pieces] = mx_codes8<T>(q[0], q[1], q[2], q[3], mx_scale_value(s));
        four |= s << (8 * k);
      }
      if ((o & 3) == 0) rs[wave * 2 + (o >> 2)][rb * 8 + i / 4] = four;
    }
    __syncthreads();
    const int t = threadIdx.x;
    if (rt * kMxPlane + t < rows) {
      uint64_t all = 0u;
#pragma unroll
      for (int k = 0; k < 8; ++k) all |= (uint64_t)reinterpret_cast<const uint8_t*>(rs[k])[t] << (8 * k);
      *reinterpret_cast<uint64_t*>(row_scales + batch * row_batch + ct * row_plane + (rt * kMxPlane + t) * 8) = all;
    }
  }
  uint8_t* out = codes + (batch * cols + (int64_t)c * N) * (deep / 2) + r0 / 2;
  auto column = [&](int j, uint32_t top, auto eight) {   // column j's codes, by eight(q, scale), and its scale
    const uint32_t s = mx_scale_of(top);
    const float f = mx_scale_value(s);
    const u32x4 w = {eight(0, f), eight(1, f), eight(2, f), eight(3, f)};
    if (col && r0 < deep) *reinterpret_cast<u32x4*>(out + (int64_t)j * (deep / 2)) = w;
    sc[(wave * 8 + o) * N + j][rb] = r0 < deep ? (uint8_t)s : 0;
  };
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if constexpr (N == 4) {
      uint32_t top = 0u;
#pragma unroll
      for (int i = 0; i < kMxBlock; ++i) top = max(top, v[i][j] & 0x7fffffffu);
      column(j, top, [&](int q, float f) {
        return mx_codes8(u32x4{v[8 * q][j], v[8 * q + 1][j], v[8 * q + 2][j], v[8 * q + 3][j]},
                         u32x4{v[8 * q + 4][j], v[8 * q + 5][j], v[8 * q + 6][j], v[8 * q + 7][j]}, f);
      });
    } else {   // two columns a word: the row pairs' low halves, then their high ones
      uint32_t m = 0u;
#pragma unroll
      for (int i = 0; i < kMxBlock; ++i) m = mx_max16(m, v[i][j]);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        auto pair = [&](int i) { return __builtin_amdgcn_perm(v[i + 1][j], v[i][j], h ? 0x07060302u : 0x05040100u); };
        column(2 * j + h, mx_f32_bits<T>(h ? m >> 16 : m & 0xffffu), [&](int q, float f) {
          return mx_codes8<T>(pair(8 * q), pair(8 * q + 2), pair(8 * q + 4), pair(8 * q + 6), f);
        });
      }
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < C; i += 64 * W) {
    const int64_t at = (int64_t)ct * C + i;
    if (at < cols)
      *reinterpret_cast<uint64_t*>(scales + batch * scale_batch + rt * plane + at * 8) = *reinterpret_cast<const uint64_t*>(sc[i]);
  }
}

// Eight values a lane, rows and planes by waves as in mx_rows_kernel (8192 x 4096 to bf16, us: a row after the other and the
// values by integer arithmetic 20, so 18.5, by the packed conversions 14.3).
template <typename T>
__global__ __launch_bounds__(kMxThreads) void mx_values_kernel(const uint32_t* __restrict__ codes, const uint8_t* __restrict__ scales,
                                                               int64_t rows, int octs, int planes, int64_t units, int64_t plane,
                                                               int64_t scale_batch, u32x4* __restrict__ out) {
  constexpr int U = kMxLoads<T>, V = Oct<T>::V;
  const int lane = threadIdx.x & 63, o = lane & 31, half = lane >> 5;
  const int64_t batch = blockIdx.y;
  codes += batch * rows * octs;
  scales += batch * scale_batch;
  out += batch * rows * octs * V;
  for (int64_t unit = (int64_t)blockIdx.x * (kMxThreads / 64) + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6); unit < units;
       unit += (int64_t)gridDim.x * (kMxThreads / 64)) {
    const int64_t rt = unit / planes, r0 = rt * 2 * U + half;
    const int at = (int)(unit - rt * planes), c = at * 32 + o;
    const bool in = c < octs;
    uint32_t w[U], s[U];
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int64_t r = r0 + 2 * i;
      const bool live = in && r < rows;
      w[i] = live ? codes[r * octs + c] : 0u;
      s[i] = live ? scales[at * plane + r * 8 + (o >> 2)] : 0u;
    }
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int64_t r = r0 + 2 * i;
      if (!in || r >= rows) continue;
      u32x4 v[V];
      mx_values8<T>(w[i], mx_scale_value(s[i]), v);
#pragma unroll
      for (int k = 0; k < V; ++k) out[(r * octs + c) * V + k] = v[k];
    }
  }
}

// Units of a wave (a plane of 2 U rows) and their workgroups for one matrix.
template <typename T> struct RowUnits {
  int octs, planes;
  int64_t units;
  dim3 grid;
  RowUnits(int64_t batch, int64_t rows, int64_t cols) {
    octs = (int)(cols / 8);
    planes = (int)mx_planes(cols);
    units = (rows + 2 * kMxLoads<T> - 1) / (2 * kMxLoads<T>) * planes;
    grid = dim3(item_grid(units, kMxThreads / 64), (unsigned)batch);
  }
};

}  // namespace

hipError_t run_mx4_rows(DType dt, const void* x, int64_t batch, int64_t rows, int64_t cols, void* codes, void* scales,
                        hipStream_t s) {
  return by_type(dt, [&](auto t) {
    const RowUnits<decltype(t)> u(batch, rows, cols);
    hipLaunchKernelGGL((mx_rows_kernel<decltype(t)>), u.grid, dim3(kMxThreads), 0, s, static_cast<const u32x4*>(x), rows, u.octs,
                       u.planes, u.units, mx_scale_rows(rows) * 8, mx_scale_bytes(rows, cols), static_cast<uint32_t*>(codes),
                       static_cast<uint8_t*>(scales));
    return hipGetLastError();
  });
}

hipError_t run_mx4_columns(DType dt, const void* x, int64_t batch, int64_t rows, int64_t cols, void* codes, void* scales,
                           void* row_codes, void* row_scales, hipStream_t s) {
  return by_type(dt, [&](auto t) {
    using T = decltype(t);
    constexpr int N = Piece<T>::N;
    const int pieces = (int)(cols / N);
    const int64_t deep = (rows + kMxBlock - 1) / kMxBlock * kMxBlock;
    auto launch = [&](auto kernel, int W) {
      const int col_tiles = (pieces + 8 * W - 1) / (8 * W);
      hipLaunchKernelGGL(kernel, dim3((unsigned)(col_tiles * mx_planes(rows)), (unsigned)batch), dim3(64 * W), 0, s,
                         static_cast<const u32x4*>(x), rows, pieces, deep, col_tiles, mx_scale_rows(cols) * 8,
                         mx_scale_bytes(cols, deep), static_cast<uint8_t*>(codes), static_cast<uint8_t*>(scales),
                         mx_scale_rows(rows) * 8, mx_scale_bytes(rows, cols), static_cast<uint32_t*>(row_codes),
                         static_cast<uint8_t*>(row_scales));
      return hipGetLastError();
    };
    if constexpr (N == 8) {
      if (row_codes) return launch(mx_columns_kernel<T, 4, true>, 4);
    }
    return launch(mx_columns_kernel<T, 1, false>, 1);
  });
}

hipError_t run_mx4_values(DType dt, const void* codes, const void* scales, int64_t batch, int64_t rows, int64_t K, void* out,
                          hipStream_t s) {
  return by_type(dt, [&](auto t) {
    const RowUnits<decltype(t)> u(batch, rows, K);
    hipLaunchKernelGGL((mx_values_kernel<decltype(t)>), u.grid, dim3(kMxThreads), 0, s, static_cast<const uint32_t*>(codes),
                       static_cast<const uint8_t*>(scales), rows, u.octs, u.planes, u.units, mx_scale_rows(rows) * 8,
                       mx_scale_bytes(rows, K), static_cast<u32x4*>(out));
    return hipGetLastError();
  });
}

}  // namespace gmlp
