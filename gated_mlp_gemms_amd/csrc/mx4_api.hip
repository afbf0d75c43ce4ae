// C-ABI of microscaled 4-bit floating point (mx4.h): argument checks, all on the host before any HIP call, the choice of
// tiles and splits, and the launches.
#include <algorithm>

#include "host_api.hpp"
#include "mx4.h"
#include "mx4.hpp"

using namespace gmlp;

namespace {

constexpr int64_t kElems = (int64_t)1 << 37;

hipStream_t stream_of(void* s) { return reinterpret_cast<hipStream_t>(s); }

mlp_status check_dtype(int dtype) {
  if (dtype != MLP_F32 && dtype != MLP_BF16 && dtype != MLP_F16)
    return fail(MLP_ERR_INVALID_ARG, "dtype %d is not an mlp_dtype", dtype);
  return MLP_OK;
}

mlp_status check_matrix(int dtype, int64_t batch, int64_t rows, int64_t cols) {
  MLP_TRY(check_dtype(dtype));
  if (batch < 0 || rows < 0 || cols < 1)
    return fail(MLP_ERR_INVALID_ARG, "batch and rows must be >= 0, columns >= 1 (%lld x %lld x %lld)", (long long)batch,
                (long long)rows, (long long)cols);
  if (batch > 65535) return fail(MLP_ERR_UNSUPPORTED, "batch is above 65535");
  if (rows > (int64_t)1 << 29) return fail(MLP_ERR_UNSUPPORTED, "rows are above 2^29");
  if (cols >= (int64_t)1 << 25) return fail(MLP_ERR_UNSUPPORTED, "columns are 2^25 or more");
  if (batch > 0 && rows > kElems / cols / batch) return fail(MLP_ERR_UNSUPPORTED, "a matrix of the problem has more than 2^37 elements");
  return MLP_OK;
}

mlp_status check_product(const linear_desc* d) {
  if (!d) return fail(MLP_ERR_INVALID_ARG, "desc is NULL");
  MLP_TRY(check_dtype(d->dtype));
  if (d->act != LINEAR_ACT_NONE && (d->act < MLP_ACT_SWIGLU || d->act > MLP_ACT_RELU))
    return fail(MLP_ERR_INVALID_ARG, "act %d is neither an mlp_act nor LINEAR_ACT_NONE", d->act);
  if (d->M < 0 || d->K < 1 || d->N < 1)
    return fail(MLP_ERR_INVALID_ARG, "M must be >= 0, K and N >= 1 (M=%lld K=%lld N=%lld)", (long long)d->M, (long long)d->K,
                (long long)d->N);
  if (d->experts < 0) return fail(MLP_ERR_INVALID_ARG, "experts = %d must be >= 0", d->experts);
  if (d->experts > MOE_MAX_EXPERTS)
    return fail(MLP_ERR_UNSUPPORTED, "E = %d experts: at most %d", d->experts, MOE_MAX_EXPERTS);
  const int64_t P = is_gated(d->act) ? 2 * d->N : d->N, E = std::max(d->experts, 1);
  if (d->M > (int64_t)1 << 29) return fail(MLP_ERR_UNSUPPORTED, "M is above 2^29");
  if (d->K >= (int64_t)1 << 25 || P >= (int64_t)1 << 25)
    return fail(MLP_ERR_UNSUPPORTED, "a leading dimension (K, N, or 2N gated) is 2^25 elements or more");
  if (d->M > kElems / P || d->M > kElems / d->K || E * P > kElems / d->K)
    return fail(MLP_ERR_UNSUPPORTED, "a matrix of the problem has more than 2^37 elements");
  if (d->K % kMxBlock) return fail(MLP_ERR_ALIGNMENT, "K must be a multiple of %d (whole blocks)", kMxBlock);
  if (d->N % 8) return fail(MLP_ERR_ALIGNMENT, "N must be a multiple of 8");
  return MLP_OK;
}

mlp_status need_rows(const void* p, int64_t elems, const char* name) {
  return elems == 0 && !p ? MLP_OK : need_ptr(p, name);
}

// ---- plans --------------------------------------------------------------------------------------

// A K-step is 256 values deep. A gated tile has half as many units as columns. Measured with forced tiles (us; 256^2, 128^2, 64^2):
// 4096 x 4096 x 11008 129, 149, 225; 4096^3 44, 47, 76; 4864 x 8192 x 2048 61, 62, 81; 2048^3 21, 12.2, 16;
// 1024 x 4096 x 4096 32, 17.8, 21.5; 512 x 4096 x 11008 34, 21, 30; 128 x 4096 x 11008 30, 15.5, 11.6; 64 x 4096 x 4096 29, 14.9,
// 8.2. 32 experts of 2048 x 1376 gate and up: 32768 rows 150, 175, 218; 8192 48, 49, 60; 4096 43, 34, 36; 1024 39, 28, 22.
struct MxTile { TileShape t; int bm, bn, slots; StepTime st; };
const MxTile kMxTiles[] = {
    {TILE_256x256, 256, 256, 1, {1.5e-6, 2.0e-6, 2.0e-6, 2.0e-6, 10e-6}},
    {TILE_128x128, 128, 128, 2, {0.50e-6, 0.69e-6, 0.85e-6, 0.99e-6, 7e-6}},
    {TILE_64x64, 64, 64, 2, {0.20e-6, 0.28e-6, 0.36e-6, 0.38e-6, 4.5e-6}},
};
const StepTime kMxWide = {0.25e-6, 0.40e-6, 0.50e-6, 0.60e-6, 5.2e-6};   // 64 x 128: 64 gated units

// Tiles of a launch, of 256 threads each: 2^32 threads are more than one can have. (With 16 x 16 tiles of few rows an expert by a
// very wide weight; larger tiles then take them.)
constexpr int64_t kMostTiles = ((int64_t)1 << 24) - 1;

struct MxPlan {
  bool skinny;       // few rows: run_mx4_skinny
  TileShape tile;
  int bm, bn;        // rows and output columns of a tile
  int splits, kps;   // parts of K, bytes of codes of one
  int tiles;         // of the launch, those of every part; 0: no tile is large enough for kMostTiles
  double est;
};

MxPlan plan_product(const linear_desc* d) {
  const bool gated = is_gated(d->act);
  const int64_t M = d->M, E = d->experts, steps = mx_planes(d->K);
  auto launched = [&](int64_t bm, int64_t bn, int64_t columns) {
    return (E ? row_tiles(M, E, bm) : (M + bm - 1) / bm) * ((columns + bn - 1) / bn);
  };
  MxPlan best{};
  best.splits = 1;
  if (M <= (E ? kMxExpertRows * E : kMxSkinnyRows) && launched(16, 16, d->N) <= kMostTiles) {
    best.skinny = true;
    best.bm = best.bn = 16;
    best.tiles = (int)launched(16, 16, d->N);
    return best;
  }
  best.est = 1e300;
  for (const MxTile& t : kMxTiles) {
    const bool wide = t.t == TILE_64x64 && gated;   // (twice the columns, for 64 gate and 64 up rows)
    // of experts: a tile each, or all their rows and half a tile each over
    const int64_t rt = E ? std::max(std::min(M, E), M / t.bm + (std::min(M, E) + 1) / 2) : (M + t.bm - 1) / t.bm;
    for (int s = 1; s <= (E ? 1 : 16); ++s) {
      const bool stacked = gated && s > 1;
      const int bn = gated && !stacked && !wide ? t.bn / 2 : t.bn;
      const int64_t N = stacked ? 2 * d->N : d->N, tiles = rt * ((N + bn - 1) / bn);
      const int64_t kps = (steps + s - 1) / s;
      if ((steps + kps - 1) / kps != s || launched(t.bm, bn, N) * s > kMostTiles) continue;
      double est = tiles_time(wide && !stacked ? kMxWide : t.st, t.slots, tiles * s, kps);
      // partial sums there and back, a launch. In 1, 2, 4, 8, 16 parts (us): 64 x 16384 x 512 on 64^2 21.7, 15.2, 11.6, 9.9, 10.1;
      // 256 x 16384 x 1024 20.6, 16.0, 13.8, 16.7, 21.9; 64 x 4096 x 4096 8.2, 9.3, 10.4, 14; 2048^3 on 128^2 12.2, 30.7, 40
      if (s > 1) est += (2.0 * s + 1.0) * (double)M * (double)N * 4.0 / 4.5e12 + 3.5e-6;
      if (est >= best.est * 0.98) continue;
      best = {false, t.t, t.bm, bn, s, (int)(kps * (kMxPlane / 2)), (int)(launched(t.bm, bn, N) * s), est};
    }
  }
  return best;
}

// A valid descriptor's plan (without rows: none is needed), and its workspace.
mlp_status make_plan(const linear_desc* d, MxPlan& p) {
  MLP_TRY(check_product(d));
  p = d->M == 0 ? MxPlan{} : plan_product(d);
  if (d->M > 0 && p.tiles == 0) return fail(MLP_ERR_UNSUPPORTED, "the product's tiles are more than 2^32 threads");
  return MLP_OK;
}
size_t workspace_of(const linear_desc* d, const MxPlan& p) {
  const int64_t P = is_gated(d->act) ? 2 * d->N : d->N;
  return p.splits > 1 ? round_up((size_t)p.splits * (size_t)d->M * (size_t)P * sizeof(float)) : kAlign;
}

}  // namespace

extern "C" {

int64_t mx4_planes(int64_t K) { return K > 0 ? mx_planes(K) : 0; }
int64_t mx4_scale_rows(int64_t rows) { return rows >= 0 ? mx_scale_rows(rows) : 0; }

mlp_status mx4_quantize(const void* x, int dtype, int64_t batch, int64_t rows, int64_t cols, void* codes, void* scales,
                        void* codes_t, void* scales_t, void* stream) {
  MLP_TRY(check_matrix(dtype, batch, rows, cols));
  const int64_t n = batch * rows;
  if ((codes == nullptr) != (scales == nullptr) && n > 0)
    return fail(MLP_ERR_INVALID_ARG, "codes and scales must both be given or both be NULL");
  if ((codes_t == nullptr) != (scales_t == nullptr) && n > 0)
    return fail(MLP_ERR_INVALID_ARG, "codes_t and scales_t must both be given or both be NULL");
  if (codes && cols % kMxBlock) return fail(MLP_ERR_ALIGNMENT, "columns must be a multiple of %d (whole blocks)", kMxBlock);
  const int q = dtype == MLP_F32 ? 4 : 8;
  if (cols % q) return fail(MLP_ERR_ALIGNMENT, "columns must be a multiple of %d (16-byte rows)", q);
  MLP_TRY(need_rows(x, n, "x"));
  for (auto& [p, name] : {std::pair<void*, const char*>{codes, "codes"}, {scales, "scales"}, {codes_t, "codes_t"}, {scales_t, "scales_t"}})
    if (p) MLP_TRY(need_ptr(p, name));
  if (n == 0) return MLP_OK;
  hipStream_t s = stream_of(stream);
  const bool both = codes && codes_t && dtype != MLP_F32;   // (8192 x 4096 of bf16: 23.5 us, in two launches 32.5)
  if (codes && !both) MLP_TRY(hip_status(run_mx4_rows(dtype_of(dtype), x, batch, rows, cols, codes, scales, s), "mx4_quantize"));
  if (codes_t)
    MLP_TRY(hip_status(run_mx4_columns(dtype_of(dtype), x, batch, rows, cols, codes_t, scales_t, both ? codes : nullptr, scales, s),
                       "mx4_quantize (transposed)"));
  return MLP_OK;
}

mlp_status mx4_dequantize(const void* codes, const void* scales, int dtype, int64_t batch, int64_t rows, int64_t K,
                          void* out, void* stream) {
  MLP_TRY(check_matrix(dtype, batch, rows, K));
  if (K % kMxBlock) return fail(MLP_ERR_ALIGNMENT, "K must be a multiple of %d (whole blocks)", kMxBlock);
  const int64_t n = batch * rows;
  MLP_TRY(need_rows(codes, n, "codes"));
  MLP_TRY(need_rows(scales, n, "scales"));
  MLP_TRY(need_rows(out, n, "out"));
  if (n == 0) return MLP_OK;
  return hip_status(run_mx4_values(dtype_of(dtype), codes, scales, batch, rows, K, out, stream_of(stream)), "mx4_dequantize");
}

size_t mx4_linear_workspace_bytes(const linear_desc* d) {
  MxPlan p;
  return make_plan(d, p) == MLP_OK ? workspace_of(d, p) : 0;
}

mlp_status mx4_linear_fwd(const linear_desc* d, const void* x, const void* x_scales, const void* w,
                          const void* w_scales, const void* w_up, const void* w_up_scales, const void* bias,
                          const void* bias_up, const void* residual, const int32_t* offsets, void* y, void* preact,
                          void* ws, size_t ws_bytes, void* stream) {
  MxPlan p;
  MLP_TRY(make_plan(d, p));
  const bool gated = is_gated(d->act);
  MLP_TRY(need_rows(x, d->M, "x"));
  MLP_TRY(need_rows(x_scales, d->M, "x_scales"));
  MLP_TRY(need_ptr(w, "w"));
  MLP_TRY(need_ptr(w_scales, "w_scales"));
  if (gated) {
    MLP_TRY(need_ptr(w_up, "w_up"));
    MLP_TRY(need_ptr(w_up_scales, "w_up_scales"));
    if ((bias == nullptr) != (bias_up == nullptr))
      return fail(MLP_ERR_INVALID_ARG, "bias and bias_up must both be given or both be NULL");
  } else {
    MLP_TRY(need_null(w_up, "w_up", "unless the activation is gated"));
    MLP_TRY(need_null(w_up_scales, "w_up_scales", "unless the activation is gated"));
    MLP_TRY(need_null(bias_up, "bias_up", "unless the activation is gated"));
  }
  if (bias) MLP_TRY(need_ptr(bias, "bias"));
  if (bias_up) MLP_TRY(need_ptr(bias_up, "bias_up"));
  if (residual) MLP_TRY(need_ptr(residual, "residual"));
  if (d->experts) MLP_TRY(need_ptr(offsets, "offsets", false));
  else MLP_TRY(need_null(offsets, "offsets", "unless desc->experts"));
  MLP_TRY(need_rows(y, d->M, "y"));
  if (preact) MLP_TRY(need_ptr(preact, "preact"));
  const size_t need = workspace_of(d, p);
  if (ws_bytes < need)
    return fail(MLP_ERR_WORKSPACE, "workspace of %zu bytes is smaller than the %zu needed", ws_bytes, need);
  MLP_TRY(need_ptr(ws, "workspace"));
  if (d->M == 0) return MLP_OK;

  hipStream_t s = stream_of(stream);
  const DType io = dtype_of(d->dtype);
  const int64_t M = d->M, N = d->N, K = d->K, P = gated ? 2 * N : N;
  Mx4Gemm a{};
  GemmArgs& g = a.g;
  g.alpha = 1.0f;
  g.act = d->act == LINEAR_ACT_NONE ? FN_NONE : act_fn_of(d->act);
  g.b_split = g.c_split = 1 << 30;
  g.M = (int)M;
  g.N = (int)N;
  g.K = (int)(K / 2);
  g.k_per_split = p.kps;
  g.A = x;
  g.B0 = w;
  g.B1 = w_up;
  g.lda = g.ldb = K / 2;
  g.C0 = y;
  g.ldc0 = N;
  g.aux = preact;
  g.ld_aux = P;
  g.half = (int)N;
  g.flags = preact ? 1 : 0;
  g.bias0 = bias;
  g.bias1 = bias_up;
  g.res = residual;
  g.ld_res = N;
  g.tiles_n = (int)(((p.splits > 1 ? P : N) + p.bn - 1) / p.bn);
  g.group_m = 8;
  a.sa = static_cast<const char*>(x_scales);
  a.sb0 = static_cast<const char*>(w_scales);
  a.sb1 = static_cast<const char*>(w_up_scales);
  a.sa_plane = mx_scale_rows(M) * 8;
  a.sb_plane = mx_scale_rows(N) * 8;
  a.offsets = offsets;
  a.experts = std::max(d->experts, 1);
  a.rows = (int)M;
  a.w_stride = N * (K / 2);
  a.ws_stride = mx_scale_bytes(N, K);
  a.bias_stride = N;
  a.splits = p.splits;
  a.tiles = p.tiles;
  if (p.splits > 1) {
    const GemmArgs join = g;
    g.N = (int)P;
    if (gated) g.b_split = (int)N;   // [w; w_up] stacked along the output columns
    g.partial = static_cast<float*>(ws);
    MLP_TRY(hip_status(run_mx4_partial(p.tile, a, s), "4-bit product (partial sums)"));
    return hip_status(run_linear_reduce(io, gated, g.partial, p.splits, join, s), "4-bit product (join)");
  }
  if (p.skinny) return hip_status(run_mx4_skinny(io, gated, a, s), "4-bit product (few rows)");
  const int epi = gated ? EPI_LIN_GATED : EPI_LIN;
  switch (io) {
    case DT_BF16: return hip_status(run_mx4_linear_bf16(epi, p.tile, a, s), "4-bit product");
    case DT_F16: return hip_status(run_mx4_linear_f16(epi, p.tile, a, s), "4-bit product");
    default: return hip_status(run_mx4_linear_f32(epi, p.tile, a, s), "4-bit product");
  }
}

}  // extern "C"
