// The linear layer's row passes: the split-K finish with its epilogue, and the backward's
// activation gradient with the bias gradient's column sums.
#include "gemm_experts.hpp"
#include "launch.hpp"

#include <algorithm>

namespace gmlp {

namespace {

constexpr int kThr = 256;

// y = res + act(sum_s partial[s] + bias), 4 columns a thread.
template <typename T, bool GATED>
__global__ __launch_bounds__(kThr) void linear_reduce_kernel(const float* __restrict__ partial, int splits,
                                                             const GemmArgs p) {
  const int n4 = p.N / 4, width = GATED ? 2 * p.N : p.N;
  const int64_t total = (int64_t)p.M * n4, slice = (int64_t)p.M * width;
  for (int64_t i = blockIdx.x * (int64_t)kThr + threadIdx.x; i < total; i += (int64_t)gridDim.x * kThr) {
    const int m = (int)(i / n4), n = (int)(i % n4) * 4;
    const float* row = partial + (int64_t)m * width + n;
    f32x4 g = *reinterpret_cast<const f32x4*>(row), u = {};
    if constexpr (GATED) u = *reinterpret_cast<const f32x4*>(row + p.N);
#pragma unroll 4
    for (int sp = 1; sp < splits; ++sp) {
      g += *reinterpret_cast<const f32x4*>(row + sp * slice);
      if constexpr (GATED) u += *reinterpret_cast<const f32x4*>(row + sp * slice + p.N);
    }
    float z[4] = {g[0], g[1], g[2], g[3]}, v[4] = {u[0], u[1], u[2], u[3]}, b[4], y[4];
    if (p.bias0) {
      Vec4<T>::load(elem_ptr<T>(p.bias0, 0, 0, n), b);
#pragma unroll
      for (int r = 0; r < 4; ++r) z[r] += b[r];
    }
    if (GATED && p.bias1) {
      Vec4<T>::load(elem_ptr<T>(p.bias1, 0, 0, n), b);
#pragma unroll
      for (int r = 0; r < 4; ++r) v[r] += b[r];
    }
    if (p.flags & 1) {
      Vec4<T>::store(elem_ptr<T>(p.aux, m, p.ld_aux, n), z);
      if constexpr (GATED) Vec4<T>::store(elem_ptr<T>(p.aux, m, p.ld_aux, p.half + n), v);
    }
    linear_act<4, GATED>(p.act, z, v, y);
    if (p.res) {
      Vec4<T>::load(elem_ptr<T>(p.res, m, p.ld_res, n), b);
#pragma unroll
      for (int r = 0; r < 4; ++r) y[r] += b[r];
    }
    Vec4<T>::store(elem_ptr<T>(p.C0, m, p.ldc0, n), y);
  }
}

// dz and its column sums over one piece of rows: 32 lanes x 8 columns across, 8 rows down. dz is rounded to T here, as
// the 16-bit operand that the matrix instructions of dx and dW take (in fp32 those products would run at a sixteenth of
// the rate): their error is about 1.4 times that of an unrounded dz. The column sums are of dz before it is rounded.
template <typename T, bool GATED>
__global__ __launch_bounds__(kThr) void linear_dact_kernel(int fn, const void* __restrict__ dy,
                                                           const void* __restrict__ preact,
                                                           const int* __restrict__ offsets, int experts, int rows,
                                                           int N, int step, void* __restrict__ dz, float* __restrict__ sums) {
  __shared__ float red[8][kDactCols];
  const int strips = (N + kDactCols - 1) / kDactCols;
  const int piece = blockIdx.x / strips, strip = blockIdx.x % strips;
  RowPiece t;
  if (!find_row_piece(offsets, experts, rows, step, [&](int total) { return piece < total ? piece : -1; }, t))
    return;
  if (t.e == experts) return;   // rows of no expert have no part in any product or sum
  const int P = GATED ? 2 * N : N;
  const int c = strip * kDactCols + (threadIdx.x & 31) * 8, rl = threadIdx.x >> 5;
  const int r0 = t.row0 + t.index * step, r1 = min(r0 + step, t.row0 + t.rows);
  const bool in0 = c < N;
  const bool half = sizeof(T) == 4 && in0 && c + 8 > N;   // fp32 widths are multiples of 4 only
  float sg[8] = {}, su[GATED ? 8 : 1] = {};
  auto load = [&](const void* p, int64_t row, int64_t ld, int col, float (&v)[8]) {
    if (half) {
      Vec4<T>::load(elem_ptr<T>(p, row, ld, col), v);
#pragma unroll
      for (int q = 4; q < 8; ++q) v[q] = 0.0f;
    } else {
      Vec8<T>::load(elem_ptr<T>(p, row, ld, col), v);
    }
  };
  auto store = [&](void* p, int64_t row, int64_t ld, int col, const float (&v)[8]) {
    if (half) Vec4<T>::store(elem_ptr<T>(p, row, ld, col), v);
    else Vec8<T>::store(elem_ptr<T>(p, row, ld, col), v);
  };
  if (in0) {
#pragma unroll 2
    for (int r = r0 + rl; r < r1; r += 8) {
      float d[8];
      load(dy, r, N, c, d);
      if (fn != FN_NONE) {
        float z[8], f[8], df[8];
        load(preact, r, P, c, z);
        linear_fn_grad<8>(fn, z, f, df);
        if constexpr (GATED) {
          float u[8], du[8];
          load(preact, r, P, N + c, u);
#pragma unroll
          for (int q = 0; q < 8; ++q) {
            du[q] = d[q] * f[q];
            d[q] *= u[q] * df[q];
            su[q] += du[q];
          }
          if (dz) store(dz, r, P, N + c, du);
        } else {
#pragma unroll
          for (int q = 0; q < 8; ++q) d[q] *= df[q];
        }
        if (dz) store(dz, r, P, c, d);
      }
#pragma unroll
      for (int q = 0; q < 8; ++q) sg[q] += d[q];
    }
  }
  if (sums == nullptr) return;
  auto join = [&](const float (&v)[8], int col0) {   // the 8 row lanes' sums, in order
#pragma unroll
    for (int q = 0; q < 8; ++q) red[rl][(threadIdx.x & 31) * 8 + q] = v[q];
    __syncthreads();
    const int n = strip * kDactCols + threadIdx.x;
    if (n < N) {
      float s = red[0][threadIdx.x];
#pragma unroll
      for (int w = 1; w < 8; ++w) s += red[w][threadIdx.x];
      sums[(int64_t)piece * P + col0 + n] = s;
    }
    __syncthreads();
  };
  join(sg, 0);
  if constexpr (GATED) join(su, N);
}

template <typename GT>
__global__ __launch_bounds__(kThr) void linear_dbias_kernel(const BiasGrad a) {
  __shared__ float red[kThr];
  bias_grad_block<GT>(a, blockIdx.x, red);
}

// The experts' partial sums joined (ExpertBwd): workgroups [0, dx_blocks) add up dx's parts (zeros behind the
// last offset), dw_blocks an expert after them the pieces of the weight gradients that have several. 4 columns a
// thread, more for many experts (of which few have pieces): a weight gradient of 4864 x 2048 f16 from 2 pieces took 95 us
// with 64 workgroups, one of 320 x 252 from 62 pieces 27 us with 20.
inline int join_blocks(int64_t elems, int experts) {
  const int64_t want = (elems / 4 + kThr - 1) / kThr;
  return (int)std::min<int64_t>(want, std::max(16, 4096 / experts));
}

template <typename T, typename GT>
__global__ __launch_bounds__(kThr) void expert_join_kernel(const ExpertBwd a, int dx_blocks, int dw_blocks) {
  const int b = blockIdx.x;
  auto add = [](const float* src, int64_t plane, int count) {
    f32x4 s = *reinterpret_cast<const f32x4*>(src);
#pragma unroll 4
    for (int i = 1; i < count; ++i) s += *reinterpret_cast<const f32x4*>(src + i * plane);
    return s;
  };
  if (b < dx_blocks) {
    const ExpertGemm& g = a.dx;
    const int kept = g.offsets ? min(max(g.offsets[g.experts], 0), g.rows) : g.rows;
    const int64_t plane = (int64_t)g.rows * g.g.N, total = plane / 4;
    for (int64_t i = b * (int64_t)kThr + threadIdx.x; i < total; i += (int64_t)dx_blocks * kThr) {
      const int64_t at = i * 4;
      const f32x4 s = at / g.g.N < kept ? add(a.part_x + at, plane, a.dx_splits) : f32x4{0.0f, 0.0f, 0.0f, 0.0f};
      const float v[4] = {s[0], s[1], s[2], s[3]};
      Vec4<T>::store(elem_ptr<T>(g.g.C0, 0, 0, at), v);
    }
    return;
  }
  const ExpertGemm& g = a.dw;
  const int e = (b - dx_blocks) / dw_blocks, part = (b - dx_blocks) % dw_blocks;
  int row0, n;
  expert_rows(g.offsets, g.experts, g.rows, e, row0, n);
  if (n <= a.piece_rows) return;
  const int slot = expert_slots_before(g.offsets, g.experts, g.rows, a.piece_rows, e);
  const int count = (n + a.piece_rows - 1) / a.piece_rows;
  if (slot + count > a.max_slots) return;   // offsets may be anything
  const int64_t plane = (int64_t)g.g.M * g.g.N, total = plane / 4;
  const float* src = a.part_w + slot * plane;
  for (int64_t i = part * (int64_t)kThr + threadIdx.x; i < total; i += (int64_t)dw_blocks * kThr) {
    const int64_t at = i * 4, m = at / g.g.N, col = at - m * g.g.N;
    const f32x4 s = add(src + at, plane, count);
    float v[4] = {s[0], s[1], s[2], s[3]};
    const bool lo = m < g.g.c_split;
    char* dst = elem_ptr<GT>(lo ? g.g.C0 : g.g.C1, lo ? m : m - g.g.c_split, g.g.ldc0, e * g.w_stride + col);
    if (g.g.accumulate) {
      float o[4];
      Vec4<float>::load(dst, o);
#pragma unroll
      for (int r = 0; r < 4; ++r) v[r] += o[r];
    }
    Vec4<GT>::store(dst, v);
  }
}

// f(type, gated) with the element type of `dt` and an integral constant.
template <typename F> hipError_t by_type(DType dt, int gated, F f) {
  auto g = [&](auto v) { return gated ? f(v, std::true_type{}) : f(v, std::false_type{}); };
  switch (dt) {
    case DT_F32: return g(float{});
    case DT_BF16: return g(bf16{});
    case DT_F16: return g(f16{});
    default: return hipErrorInvalidValue;
  }
}

}  // namespace

hipError_t run_linear_reduce(DType io, int gated, const float* partial, int splits, const GemmArgs& a, hipStream_t s) {
  const int64_t items = (int64_t)a.M * (a.N / 4);
  const dim3 grid((unsigned)std::min<int64_t>((items + kThr - 1) / kThr, 256 * 64));
  return by_type(io, gated, [&](auto v, auto g) {
    hipLaunchKernelGGL((linear_reduce_kernel<decltype(v), decltype(g)::value>), grid, dim3(kThr), 0, s, partial, splits, a);
    return hipGetLastError();
  });
}

hipError_t run_linear_dact(DType io, int gated, int fn, const void* dy, const void* preact, const int* offsets,
                           int experts, int64_t rows, int64_t N, void* dz, float* sums, hipStream_t s) {
  const dim3 grid((unsigned)(dact_pieces(rows, N, experts) * ((N + kDactCols - 1) / kDactCols)));
  return by_type(io, gated, [&](auto v, auto g) {
    hipLaunchKernelGGL((linear_dact_kernel<decltype(v), decltype(g)::value>), grid, dim3(kThr), 0, s, fn, dy, preact,
                       offsets, experts, (int)rows, (int)N, dact_rows(rows, N), dz, sums);
    return hipGetLastError();
  });
}

hipError_t run_linear_dbias(DType io, const BiasGrad& a, hipStream_t s) {
  return by_type(a.accumulate ? DT_F32 : io, 0, [&](auto v, auto) {
    hipLaunchKernelGGL((linear_dbias_kernel<decltype(v)>), dim3(a.grid), dim3(kThr), 0, s, a);
    return hipGetLastError();
  });
}

hipError_t run_expert_join(DType io, const ExpertBwd& a, hipStream_t s) {
  const int64_t items = a.dx_splits > 1 ? (int64_t)a.dx.rows * a.dx.g.N / 4 : 0;
  const int dx_blocks = (int)std::min<int64_t>((items + kThr - 1) / kThr, 256 * 16);
  const int dw_blocks = a.piece_rows ? join_blocks((int64_t)a.dw.g.M * a.dw.g.N, a.dw.experts) : 0;
  const int blocks = dx_blocks + a.dw.experts * dw_blocks;
  if (blocks == 0) return hipSuccess;
  return by_type(io, a.dw.g.accumulate, [&](auto v, auto acc) {
    using T = decltype(v);
    using GT = typename std::conditional<decltype(acc)::value, float, T>::type;
    hipLaunchKernelGGL((expert_join_kernel<T, GT>), dim3(blocks), dim3(kThr), 0, s, a, dx_blocks, dw_blocks);
    return hipGetLastError();
  });
}

}  // namespace gmlp
