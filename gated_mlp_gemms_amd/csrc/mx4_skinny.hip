// Products of microscaled 4-bit operands with few rows (mx4.h): decode-size token counts, one weight or one an expert.
// Bound by the weights' bytes, 17 / 32 of one an element: a wave streams 16 rows of the weight and multiplies them, 128 values at
// a time, with 16 tokens (v_mfma_scale_f32_16x16x128_f8f6f4, weights as A). The four waves of a workgroup take every
// fourth step of 256 values, so that most bytes of a problem like 4096 x 11008 are under way at once, and
// join their sums through LDS in order. In a step a lane has 32 bytes of its row, two blocks that follow one another, so a
// product's scale is one byte of the two that the lane loads.
#include "gemm_experts.hpp"
#include "launch.hpp"
#include "mx4.hpp"

namespace gmlp {

namespace {

struct MxStep {   // a lane's share of one row's 256 values
  u32x4 lo, hi;
  uint32_t s;
};

template <int S>
__device__ __forceinline__ void mx_mma16(const u32x4& a, const u32x4& b, uint32_t sa, uint32_t sb, f32x4& acc) {
  const i32x8 av = {(int)a[0], (int)a[1], (int)a[2], (int)a[3], 0, 0, 0, 0};
  const i32x8 bv = {(int)b[0], (int)b[1], (int)b[2], (int)b[3], 0, 0, 0, 0};
  acc = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(av, bv, acc, 4, 4, S, (int)sa, S, (int)sb);   // 4: e2m1
}

constexpr int kWaves = 4;

// U steps under way at once. One weight: 1, the registers of few steps leave room for more waves (us, 1 and 4 steps: 16 rows of
// 4096 x 11008 8.9 and 9.0, of 11008 x 4096 8.2 and 8.8, one row 6.7 and 7.0; with 2 waves 12.0 of 11008 x 4096, with 8 8.3, with 32
// weight rows a wave 11.7). Experts: 4, fewer waves go through fewer places in memory at once (96 rows of 36 experts of
// 2048 x 1376 gate and up 25.9 and 23.9, 4.5 TB/s; 48 of 29 19.8 and 18.7).
template <typename IoT, bool GATED, int U>
__global__ __launch_bounds__(64 * kWaves) void mx_skinny_kernel(const Mx4Gemm a) {
  constexpr int G = GATED ? 2 : 1, W = kWaves;
  __shared__ f32x4 red[W][G][64];
  const GemmArgs& g = a.g;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r = lane & 15, q = lane >> 4;
  const int tiles_n = g.tiles_n, tile = (int)blockIdx.x / tiles_n, n0 = ((int)blockIdx.x - tile * tiles_n) * 16;

  RowPiece t;
  if (a.offsets == nullptr) {
    t = {0, 0, a.rows, tile, 0};
  } else if (!find_row_piece(a.offsets, a.experts, a.rows, 16, [&](int total) { return tile < total ? tile : -1; }, t)) {
    return;
  }
  const int row0 = t.row0 + t.index * 16, rows = min(t.rows - t.index * 16, 16);
  const bool none = t.e == a.experts;   // rows of no expert: zeros (plus the residual)

  f32x4 acc[G];
#pragma unroll
  for (int k = 0; k < G; ++k) acc[k] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  if (!none) {
    const int steps = (g.K + 127) / 128, full = g.K / 128;
    const int64_t wrow = min(n0 + r, g.N - 1);
    const char* w[G];
    const char* ws[G];
#pragma unroll
    for (int k = 0; k < G; ++k) {
      w[k] = static_cast<const char*>(k == 0 ? g.B0 : g.B1) + t.e * a.w_stride + wrow * g.ldb + q * 32;
      ws[k] = (k == 0 ? a.sb0 : a.sb1) + t.e * a.ws_stride + wrow * 8 + q * 2;
    }
    const int64_t row = row0 + min(r, rows - 1);
    const char* x = static_cast<const char*>(g.A) + row * g.lda + q * 32;
    const char* xs = a.sa + row * 8 + q * 2;
    // step s of a row; past the last whole step what lies behind the row is zeros
    auto load = [&](const char* p, const char* ps, int64_t plane, int s, auto whole) {
      MxStep v;
      if constexpr (decltype(whole)::value) {
        v.lo = *reinterpret_cast<const u32x4*>(p + s * 128);
        v.hi = *reinterpret_cast<const u32x4*>(p + s * 128 + 16);
        v.s = *reinterpret_cast<const uint16_t*>(ps + s * plane);
      } else {
        const u32x4 zero = {0u, 0u, 0u, 0u};
        const int at = s * 128 + q * 32;
        v.lo = at < g.K ? *reinterpret_cast<const u32x4*>(p + s * 128) : zero;
        v.hi = at + 16 < g.K ? *reinterpret_cast<const u32x4*>(p + s * 128 + 16) : zero;
        v.s = s < steps ? *reinterpret_cast<const uint16_t*>(ps + s * plane) : 0u;
      }
      return v;
    };
    auto turn = [&](int s0, auto whole, auto count) {
      constexpr int UU = decltype(count)::value;
      MxStep vw[UU][G], vx[UU];
#pragma unroll
      for (int u = 0; u < UU; ++u) {
#pragma unroll
        for (int k = 0; k < G; ++k) vw[u][k] = load(w[k], ws[k], a.sb_plane, s0 + u * W, whole);
        vx[u] = load(x, xs, a.sa_plane, s0 + u * W, whole);
      }
#pragma unroll
      for (int u = 0; u < UU; ++u)
#pragma unroll
        for (int k = 0; k < G; ++k) {
          mx_mma16<0>(vw[u][k].lo, vx[u].lo, vw[u][k].s, vx[u].s, acc[k]);
          mx_mma16<1>(vw[u][k].hi, vx[u].hi, vw[u][k].s, vx[u].s, acc[k]);
        }
    };
    int s0 = wave;
    for (; s0 + (U - 1) * W < full; s0 += U * W) turn(s0, std::true_type{}, std::integral_constant<int, U>{});
    for (; s0 < steps; s0 += W) turn(s0, std::false_type{}, std::integral_constant<int, 1>{});
  }
#pragma unroll
  for (int k = 0; k < G; ++k) red[wave][k][lane] = acc[k];
  __syncthreads();

  // a lane of the product has token l % 16 and 4 columns from 4 (l / 16) on
  const int n = n0 + 4 * q;
  if (wave != 0 || r >= rows || n >= g.N) return;
  const int64_t row = row0 + r;
  float v[4] = {}, u[4] = {}, y[4] = {};
  if (!none) {
#pragma unroll
    for (int s = 0; s < W; ++s) {
      const f32x4 z = red[s][0][lane], z1 = red[s][G - 1][lane];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[i] += z[i];
        if constexpr (GATED) u[i] += z1[i];
      }
    }
    auto bias = [&](const void* b, float (&z)[4]) {
      if (b == nullptr) return;
      float f[4];
      Vec4<IoT>::load(elem_ptr<IoT>(b, t.e, a.bias_stride, n), f);
#pragma unroll
      for (int i = 0; i < 4; ++i) z[i] += f[i];
    };
    bias(g.bias0, v);
    if constexpr (GATED) bias(g.bias1, u);
  }
  if (g.flags & 1) {
    Vec4<IoT>::store(elem_ptr<IoT>(g.aux, row, g.ld_aux, n), v);
    if constexpr (GATED) Vec4<IoT>::store(elem_ptr<IoT>(g.aux, row, g.ld_aux, g.half + n), u);
  }
  if (!none) linear_act<4, GATED>(g.act, v, u, y);
  if (g.res) {
    float o[4];
    Vec4<IoT>::load(elem_ptr<IoT>(g.res, row, g.ld_res, n), o);
#pragma unroll
    for (int i = 0; i < 4; ++i) y[i] += o[i];
  }
  Vec4<IoT>::store(elem_ptr<IoT>(g.C0, row, g.ldc0, n), y);
}

template <typename IoT, bool GATED> hipError_t launch(const Mx4Gemm& a, hipStream_t s) {
  if (a.offsets == nullptr) hipLaunchKernelGGL((mx_skinny_kernel<IoT, GATED, 1>), dim3(a.tiles), dim3(64 * kWaves), 0, s, a);
  else hipLaunchKernelGGL((mx_skinny_kernel<IoT, GATED, 4>), dim3(a.tiles), dim3(64 * kWaves), 0, s, a);
  return hipGetLastError();
}

}  // namespace

hipError_t run_mx4_skinny(DType io, int gated, const Mx4Gemm& a, hipStream_t s) {
  switch (io) {
    case DT_BF16: return gated ? launch<bf16, true>(a, s) : launch<bf16, false>(a, s);
    case DT_F16: return gated ? launch<f16, true>(a, s) : launch<f16, false>(a, s);
    default: return gated ? launch<float, true>(a, s) : launch<float, false>(a, s);
  }
}

}  // namespace gmlp
