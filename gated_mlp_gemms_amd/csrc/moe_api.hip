// C-ABI of the mixture-of-experts operators (moe.h): argument checks, all on the host before any HIP
// call, the choice of tiles and splits, and the launches.
#include <algorithm>
#include <math.h>

#include "host_api.hpp"
#include "moe.h"

using namespace gmlp;

namespace {

constexpr int64_t kRowLimit = (int64_t)1 << 30;

mlp_status check_dtype(int dtype) {
  if (dtype != MLP_F32 && dtype != MLP_BF16 && dtype != MLP_F16)
    return fail(MLP_ERR_INVALID_ARG, "dtype %d is not an mlp_dtype", dtype);
  return MLP_OK;
}

// A tensor of `elems` elements: may be NULL when it has none.
mlp_status need_buf(const void* p, int64_t elems, const char* name, bool align16 = true) {
  return elems == 0 && !p ? MLP_OK : need_ptr(p, name, align16);
}

mlp_status check_experts(int64_t E) {
  if (E < 1) return fail(MLP_ERR_INVALID_ARG, "E = %lld experts: at least 1", (long long)E);
  if (E > MOE_MAX_EXPERTS)
    return fail(MLP_ERR_UNSUPPORTED, "E = %lld experts: at most %d", (long long)E, MOE_MAX_EXPERTS);
  return MLP_OK;
}

mlp_status check_choices(int64_t T, int64_t E, int64_t k) {
  MLP_TRY(check_experts(E));
  if (T < 0) return fail(MLP_ERR_INVALID_ARG, "T = %lld tokens", (long long)T);
  if (k < 1 || k > E) return fail(MLP_ERR_INVALID_ARG, "k = %lld is not in [1, E = %lld]", (long long)k, (long long)E);
  if (k > MOE_MAX_CHOICES)
    return fail(MLP_ERR_UNSUPPORTED, "k = %lld choices a token: at most %d", (long long)k, MOE_MAX_CHOICES);
  if (T > kRowLimit / k) return fail(MLP_ERR_UNSUPPORTED, "T k is above 2^30");
  return MLP_OK;
}

mlp_status check_router(int dtype, int64_t T, int64_t E, int64_t k, int score, int renorm) {
  MLP_TRY(check_dtype(dtype));
  MLP_TRY(check_choices(T, E, k));
  if (score != MOE_SOFTMAX && score != MOE_SIGMOID)
    return fail(MLP_ERR_INVALID_ARG, "score %d is not a moe_score", score);
  if (renorm != 0 && renorm != 1) return fail(MLP_ERR_INVALID_ARG, "renorm must be 0 or 1");
  return MLP_OK;
}

mlp_status check_rows(int dtype, int64_t T, int64_t E, int64_t k, int64_t d) {
  MLP_TRY(check_dtype(dtype));
  MLP_TRY(check_choices(T, E, k));
  if (d < 1) return fail(MLP_ERR_INVALID_ARG, "d = %lld must be >= 1", (long long)d);
  if (d >= (int64_t)1 << 25) return fail(MLP_ERR_UNSUPPORTED, "d is 2^25 or more");
  const int q = dtype == MLP_F32 ? 4 : 8;
  if (d % q) return fail(MLP_ERR_ALIGNMENT, "d must be a multiple of %d (16-byte rows)", q);
  return MLP_OK;
}

hipStream_t stream_of(void* s) { return reinterpret_cast<hipStream_t>(s); }
int pieces_of(int dtype, int64_t d) { return (int)(d * esize(dtype) / 16); }

// ---- linear layer -------------------------------------------------------------------------------

mlp_status check_linear(const linear_desc* d) {
  if (!d) return fail(MLP_ERR_INVALID_ARG, "desc is NULL");
  MLP_TRY(check_dtype(d->dtype));
  if (d->act != LINEAR_ACT_NONE && (d->act < MLP_ACT_SWIGLU || d->act > MLP_ACT_RELU))
    return fail(MLP_ERR_INVALID_ARG, "act %d is neither an mlp_act nor LINEAR_ACT_NONE", d->act);
  if (d->M < 0 || d->K < 1 || d->N < 1)
    return fail(MLP_ERR_INVALID_ARG, "M must be >= 0, K and N >= 1 (M=%lld K=%lld N=%lld)", (long long)d->M,
                (long long)d->K, (long long)d->N);
  if (d->experts < 0) return fail(MLP_ERR_INVALID_ARG, "experts = %d must be >= 0", d->experts);
  if (d->experts > 0) MLP_TRY(check_experts(d->experts));
  const int64_t P = is_gated(d->act) ? 2 * d->N : d->N, E = std::max(d->experts, 1), lim = (int64_t)1 << 37;
  if (d->M > kRowLimit / 2) return fail(MLP_ERR_UNSUPPORTED, "M is above 2^29");
  if (d->K >= (int64_t)1 << 25 || d->N >= (int64_t)1 << 25 || P >= (int64_t)1 << 25)
    return fail(MLP_ERR_UNSUPPORTED, "a leading dimension (K, N, or 2N gated) is 2^25 elements or more");
  if (d->M > lim / P || d->M > lim / d->K || E * P > lim / d->K)
    return fail(MLP_ERR_UNSUPPORTED, "a matrix of the problem has more than 2^37 elements");
  if ((d->M / kDactRowsFew + 1) * (E + 1) >= (int64_t)1 << 31)
    return fail(MLP_ERR_UNSUPPORTED, "M times experts is above 2^35");
  const int q = d->dtype == MLP_F32 ? 4 : 8;
  if (d->K % q || d->N % q) return fail(MLP_ERR_ALIGNMENT, "K and N must be multiples of %d (16-byte rows)", q);
  return MLP_OK;
}

GemmArgs linear_args(const linear_desc* d) {
  GemmArgs a{};
  a.alpha = 1.0f;
  a.act = d->act == LINEAR_ACT_NONE ? FN_NONE : act_fn_of(d->act);
  a.b_split = 1 << 30;
  a.c_split = 1 << 30;
  return a;
}

// The tile shapes of the linear layer's and the experts' products. The 16-bit ones' rates are plan_gemm's;
// 64 x 64: as measured in step_time. fp32 (of its own, a sixteenth of the 16-bit peak): 104-127 of 154 TFLOP/s at 128 x 128.
// A gated fp32 tile has 64 units in either shape, and by step_time the one of 64 rows is faster at every size.
int linear_tiles(DType in, bool gated, TileInfo (&t)[4]) {
  int n = 0;
  if (in == DT_F32) {
    if (!gated) t[n++] = {TILE_128x128_RING, 128, 128, 2, 0.85};
    t[n++] = {TILE_64x64, 64, gated ? 128 : 64, 2, 0.70};
    return n;
  }
  for (const TileInfo& i : kTiles)
    if (i.t == TILE_256x256_W8 || i.t == TILE_256x128_W8 || i.t == TILE_128x128) t[n++] = i;
  t[n++] = {TILE_64x64, 64, gated ? 128 : 64, 2, gated ? 0.26 : 0.20};
  return n;
}

// StepTime of a tile, a K-step 64 deep (fp32 32). Measured with forced tiles (us): 2000^3 128 x 128 (one a CU) 26.3, 256 x 128
// (128 tiles) 33.6, 64 x 64 (two rounds) 38.8; 2000 x 512 x 4096 gated 24.1 / 30.9 / 30.1 / 37.2 (256 x 256, 256 x 128, 128 x 128,
// 64 x 128); 1000 x 4096 x 512 73 / 47 / 38 / 22; a weight gradient of 2440 x 1560 over 14050 rows in 260 tiles of 128 x 128,
// two on 4 CUs, 211 (256 x 256 in three parts of K 125), one of 2048 x 2048 over 8192 in 256 of them 74.
StepTime step_time(TileShape t, DType in, bool gated) {
  if (in == DT_F32) {
    if (t != TILE_64x64) return {2.2e-6, 2.3e-6, 4.2e-6, 4.5e-6, 5e-6};
    return gated ? StepTime{1.0e-6, 1.2e-6, 1.9e-6, 2.1e-6, 2e-6} : StepTime{0.55e-6, 0.65e-6, 0.95e-6, 1.1e-6, 2e-6};
  }
  switch (t) {
    case TILE_256x256_W8: return {1.05e-6, 1.95e-6, 1.95e-6, 1.95e-6, 4e-6};
    case TILE_256x128_W8: return {0.66e-6, 1.07e-6, 1.07e-6, 1.07e-6, 3.5e-6};
    case TILE_128x128: return {0.50e-6, 0.65e-6, 0.95e-6, 1.20e-6, 2.5e-6};
    default: return gated ? StepTime{0.33e-6, 0.55e-6, 0.60e-6, 0.77e-6, 1.5e-6} : StepTime{0.25e-6, 0.40e-6, 0.42e-6, 0.52e-6, 1.5e-6};
  }
}

Plan plan_linear_gemm(DType in, int64_t M, int64_t N, int64_t K, bool allow_split, bool gated) {
  TileInfo t[4];
  const int n = linear_tiles(in, gated, t), bk = bk_of(in);
  Plan best{};
  best.est = 1e300;
  for (int i = 0; i < n; ++i) {
    const StepTime st = step_time(t[i].t, in, gated);
    const int64_t units = gated ? t[i].bn / 2 : t[i].bn;
    const int64_t tm = (M + t[i].bm - 1) / t[i].bm, tn = (N + units - 1) / units;
    for (int s = 1; s <= (allow_split ? 16 : 1); ++s) {
      const int64_t kps = ((K + s - 1) / s + bk - 1) / bk * bk;
      if ((K + kps - 1) / kps != s) continue;
      double est = tiles_time(st, t[i].slots, tm * tn * s, kps / bk);
      if (s > 1) est += (2.0 * s * M * N * 4.0 + M * N * 4.0) / 6.0e12 + 4e-6;   // partial sums there and back, a launch
      if (est >= best.est * 0.98) continue;
      best.est = est;
      best.tile = t[i].t;
      best.splits = s;
      best.k_per_split = (int)kps;
      best.tiles_m = (int)tm;
      best.tiles_n = (int)tn;
      best.group_m = tn == 3 ? 1 : (int)std::min<int64_t>(tm, 8);   // as plan_tiles
      best.grid = (int)(tm * tn * s);
    }
  }
  return best;
}

// Forward with one weight: the fused product, or split along K into fp32 partials that
// run_linear_reduce finishes (gated: of the stacked [g | u]); whichever the time model prefers.
struct LinearFwd {
  bool skinny;
  Plan plan;   // splits > 1: partial sums over [M, P]
};
LinearFwd plan_linear(const linear_desc* d) {
  LinearFwd f{};
  const DType io = dtype_of(d->dtype);
  const bool gated = is_gated(d->act);
  f.skinny = io != DT_F32 && d->M <= kSkinnyMaxRows;
  if (f.skinny || d->M == 0) return f;
  f.plan = plan_linear_gemm(io, d->M, d->N, d->K, false, gated);
  if (gated && d->N % 8) return f;   // the stacked operand changes matrices at a multiple of 8 rows only
  const Plan split = plan_linear_gemm(io, d->M, gated ? 2 * d->N : d->N, d->K, true, false);
  if (split.splits > 1 && split.est < f.plan.est) f.plan = split;
  return f;
}

// The experts' products: the streaming kernel for a few rows an expert, else tiles.
enum ExpertForm { EXPERT_SKINNY, EXPERT_TILES };
struct ExpertPlan {
  ExpertForm form;
  TileShape tile;
  int bm, bn;
  double est;            // seconds
  // backward: parts of dx's K, rows of a weight gradient's piece (0: whole experts) and the partial sums'
  // slots that those take at most
  int dx_splits, piece_rows, max_slots;
  bool dw_first;
  int strip_parts;       // backward, few rows an expert: shares of a strip's weight gradient (ExpertBwd); else 0
};

// K-steps that are not worth another launch to join them (about 0.3 us each of a product with CUs to spare, against 5 us).
constexpr double kJoinSteps = 20.0;

// The backward with few rows an expert: dx in 64 x 128 tiles, the weight gradients in strips.
ExpertPlan plan_experts_few(const linear_desc* d) {
  const int64_t M = d->M, E = std::max(d->experts, 1), P = is_gated(d->act) ? 2 * d->N : d->N;
  const int bk = bk_of(dtype_of(d->dtype)), slots = 512;
  ExpertPlan p{EXPERT_TILES, TILE_128x128, 64, 128, 0.0, 1, 0, 0, false, 0};
  const int64_t tiles_m = (P + kStripTileM - 1) / kStripTileM, strips = E * ((d->K + kStripTileN - 1) / kStripTileN);
  p.strip_parts = (int)std::min<int64_t>(tiles_m, std::max<int64_t>(1, 2 * slots / strips));
  const int64_t kx = (P + bk - 1) / bk, tx = (M / 64 + (std::min(M, E) + 1) / 2) * ((d->K + 127) / 128);
  const double work = ((double)tx * (kx + 2) + (double)(strips * tiles_m) * ((double)(M / E) / bk + 1)) / slots;
  while (p.dx_splits < 16 && kx / p.dx_splits > std::max(kJoinSteps, work) && kx / (p.dx_splits + 1) >= 8) ++p.dx_splits;
  const int64_t piece = (int64_t)std::max(kJoinSteps, work) * bk;   // for an expert that most rows go to
  if (M >= piece + piece / 2) {
    p.piece_rows = (int)piece;
    p.max_slots = (int)(2 * (M / piece) + 1);
  }
  const int es = esize(d->dtype);
  p.est = 4e-6 + (2.0 * (double)E * P + (double)M) * (double)d->K * es / 5.0e12 + (p.dx_splits > 1 || p.piece_rows ? 4e-6 : 0.0);
  return p;
}

// The tile by the time model of step_time, every expert ending in half a row tile on average: forward
// [M, K] -> [M, N], or backward both products ([M, P] -> [M, K], and K over the expert's rows).
ExpertPlan plan_experts(const linear_desc* d, bool fwd) {
  const DType io = dtype_of(d->dtype);
  const bool gated = is_gated(d->act);
  const int64_t M = d->M, E = std::max(d->experts, 1), P = gated ? 2 * d->N : d->N;
  if (fwd && io != DT_F32 && M <= kExpertFewRows * E) return {EXPERT_SKINNY, TILE_128x128, 128, 128, 0.0, 1, 0, 0, false, 0};
  if (!fwd && io != DT_F32 && M <= E * (E * P * d->K * 2 < kStreamGradBytes ? kStripRowsSmall : kStripRows)) return plan_experts_few(d);
  TileInfo t[4];
  const int n = linear_tiles(io, fwd && gated, t), bk = bk_of(io);
  ExpertPlan best{EXPERT_TILES, TILE_COUNT, 0, 0, 1e300, 1, 0, 0, false, 0};
  for (int i = 0; i < n; ++i) {
    if (t[i].t == TILE_256x128_W8) continue;
    const StepTime st = step_time(t[i].t, io, fwd && gated);
    const int64_t bnc = fwd && gated ? t[i].bn / 2 : t[i].bn, slots = 256 * t[i].slots;
    const int64_t rt = std::max<int64_t>(1, M / t[i].bm + (std::min(M, E) + 1) / 2);
    const int64_t kx = ((fwd ? d->K : P) + bk - 1) / bk;
    const int64_t tx = rt * (((fwd ? d->N : d->K) + bnc - 1) / bnc);
    ExpertPlan p{EXPERT_TILES, t[i].t, t[i].bm, t[i].bn, 0.0, 1, 0, 0, false, 0};
    if (fwd) {
      p.est = tiles_time(st, t[i].slots, tx, kx);
    } else {
      const int64_t tw = (P + t[i].bm - 1) / t[i].bm * ((d->K + t[i].bn - 1) / t[i].bn);   // tiles an expert
      const int64_t kw = (M / E + bk - 1) / bk;
      const double work = ((double)tx * (kx + 2) + (double)E * tw * (kw + 2)) / slots;   // K-steps a slot
      // dx in parts while a part is longer than half of what a slot has to do, and takes 8 K-steps
      const double least = io == DT_F32 ? 8.0 : kJoinSteps;
      while (p.dx_splits < 16 && kx / p.dx_splits > std::max(least, work) && kx / (p.dx_splits + 1) >= 8) ++p.dx_splits;
      // weight gradients over pieces of the rows: with few tiles of half a slot's work, else of all of it
      // (an expert that most rows go to)
      const int64_t piece = (int64_t)std::max(least, E * tw < 2 * slots ? work / 2 : work) * bk;
      int64_t kd = std::min<int64_t>((M + bk - 1) / bk, E == 1 ? (M + bk - 1) / bk : 2 * kw);   // longest tile expected
      if (M >= piece + piece / 2) {
        p.piece_rows = (int)piece;
        p.max_slots = (int)std::min<int64_t>(2 * (M / piece) + 1, (int64_t)1 << 30);
        kd = std::min(kd, piece / bk);
      }
      p.dw_first = kd > kx / p.dx_splits;
      // seconds: what a slot does in all, and the longest tile
      const double items = (double)tx * p.dx_splits + (double)E * tw;
      const double busy = std::min(1.0, items / slots), step = items <= 256.0 ? st.few + (st.one - st.few) * items / 256.0
                                                                            : st.one + (st.full - st.one) * busy;
      const double all = (((double)tx * kx + (double)E * tw * kw) * step + items * st.rest) / slots;
      const double longest = (double)std::max<int64_t>(kx / p.dx_splits, kd) * step + st.rest;
      p.est = std::max(longest, all + longest / 4);
      if (p.dx_splits > 1) p.est += ((double)p.dx_splits * 2 + 1) * (double)M * (double)d->K * 4.0 / 6.0e12;
      if (p.piece_rows && E == 1) p.est += ((double)(M / piece + 1) * 2 + 1) * (double)P * (double)d->K * 4.0 / 6.0e12;
      if (p.dx_splits > 1 || p.piece_rows) p.est += 4e-6;
    }
    if (p.est < best.est * 0.98) best = p;
  }
  return best;
}

// The backward's launches.
struct LinearBwd {
  bool small;          // dx, dW and the bias gradient in one launch, as one expert's
  bool group;          // dx and dW in one launch of 8-wave 256 x 256 tiles (16-bit)
  Plan gdx, gdw;
  RowsPlan dx;
  Plan dw;
};
LinearBwd plan_linear_bwd(const linear_desc* d, bool dx, bool dw) {
  LinearBwd b{};
  const DType io = dtype_of(d->dtype);
  const int64_t P = is_gated(d->act) ? 2 * d->N : d->N;
  if (io == DT_F32) b.dx.main = plan_linear_gemm(io, d->M, d->K, P, true, false);
  else b.dx = plan_rows(io, d->M, d->K, P);
  b.dw = plan_linear_gemm(io, P, d->K, d->M, true, false);
  // each launch counts for 4 us: small products take fewer
  const double apart = (dx ? (b.dx.m1 ? b.dx.main.est + b.dx.tail.est : b.dx.main.est) + 4e-6 : 0.0) +
                       (dw ? b.dw.est + 4e-6 : 0.0);
  // (fp32, whose launches are modelled a little short: 10000 x 300 x 500 89 us in one, 101 apart)
  b.small = dx && dw && plan_experts(d, false).est + 4e-6 < (io == DT_F32 ? 1.05 : 0.97) * apart;
  if (b.small || !dx || !dw || io == DT_F32) return b;
  b.gdx = plan_gemm(io, d->M, d->K, P, false, false, TILE_256x256_W8);
  b.gdw = plan_gemm(io, P, d->K, d->M, false, false, TILE_256x256_W8);
  const int64_t tiles[2] = {b.gdx.grid, b.gdw.grid}, steps[2] = {(P + 63) / 64, (d->M + 63) / 64};
  const int64_t t2[2] = {tiles[steps[0] >= steps[1] ? 0 : 1], tiles[steps[0] >= steps[1] ? 1 : 0]};
  const int64_t s2[2] = {std::max(steps[0], steps[1]), std::min(steps[0], steps[1])};
  if (tiles[0] > 32 * 256 || tiles[1] > 32 * 256) return b;   // many rounds: nothing to fill
  const TileInfo& w8 = kTiles[0];
  const double t_group = list_makespan(t2, s2, 2, 1.0) * (2.0 * w8.bm * w8.bn * 64 / (w8.eff * 9.83e12));
  b.group = t_group + 4e-6 < 0.97 * apart;
  return b;
}

struct LinearWs { size_t dz, sums, partial, part_w, total; };
LinearWs linear_ws(const linear_desc* d, int phase) {
  LinearWs w{};
  const int64_t P = is_gated(d->act) ? 2 * d->N : d->N, E = std::max(d->experts, 1);
  size_t at = 0;
  auto take = [&](size_t& off, size_t bytes) { off = at; at += round_up(bytes); };
  if (phase == LINEAR_FWD) {
    const LinearFwd f = d->experts ? LinearFwd{} : plan_linear(d);
    take(w.partial, partial_bytes(f.plan, d->M, P));
  } else {
    take(w.dz, d->act == LINEAR_ACT_NONE ? 0 : (size_t)d->M * P * esize(d->dtype));
    take(w.sums, (size_t)dact_pieces(d->M, d->N, E) * P * sizeof(float));
    const LinearBwd b = d->experts || d->M == 0 ? LinearBwd{} : plan_linear_bwd(d, true, true);
    const ExpertPlan p = plan_experts(d, false);
    const bool one = d->experts || b.small;
    take(w.partial, std::max({d->experts || d->M == 0 ? 0 : std::max(partial_bytes(b.dx, d->M, d->K), partial_bytes(b.dw, P, d->K)),
                              one && p.dx_splits > 1 ? (size_t)p.dx_splits * d->M * d->K * sizeof(float) : 0}));
    take(w.part_w, one ? (size_t)p.max_slots * P * d->K * sizeof(float) : 0);
  }
  w.total = std::max<size_t>(at, kAlign);
  return w;
}

mlp_status check_linear_ws(const linear_desc* d, int phase, const void* ws, size_t ws_bytes) {
  const size_t need = linear_ws(d, phase).total;
  if (ws_bytes < need)
    return fail(MLP_ERR_WORKSPACE, "workspace of %zu bytes is smaller than the %zu needed", ws_bytes, need);
  return need_ptr(ws, "workspace");
}

// The arguments of both directions that are checked alike.
mlp_status check_weights(const linear_desc* d, const void* x, const void* w, const void* w_up, const int32_t* offsets) {
  MLP_TRY(need_buf(x, d->M * d->K, "x"));
  MLP_TRY(need_ptr(w, "w"));
  if (is_gated(d->act)) MLP_TRY(need_ptr(w_up, "w_up"));
  else MLP_TRY(need_null(w_up, "w_up", "unless the activation is gated"));
  if (d->experts) return need_ptr(offsets, "offsets", false);
  return need_null(offsets, "offsets", "unless desc->experts");
}

ExpertGemm expert_gemm(const linear_desc* d, const GemmArgs& g, const int32_t* offsets) {
  ExpertGemm e{};
  e.g = g;
  e.offsets = offsets;
  e.experts = std::max(d->experts, 1);
  e.rows = (int)d->M;
  e.w_stride = d->N * d->K;
  e.bias_stride = d->N;
  return e;
}

}  // namespace

extern "C" {

int moe_abi_version(void) { return 1; }

mlp_status moe_route(const void* logits, int dtype, int64_t T, int64_t E, int64_t k, int score, int renorm,
                     int32_t* ids, float* weights, void* stream) {
  MLP_TRY(check_router(dtype, T, E, k, score, renorm));
  MLP_TRY(need_buf(logits, T, "logits"));
  MLP_TRY(need_buf(ids, T, "ids", false));
  MLP_TRY(need_buf(weights, T, "weights", false));
  if (T == 0) return MLP_OK;
  return hip_status(run_moe_route(dtype_of(dtype), logits, T, (int)E, (int)k, score == MOE_SIGMOID, renorm, ids, weights,
                                  stream_of(stream)), "moe_route");
}

mlp_status moe_route_bwd(const void* logits, const int32_t* ids, const float* dweights, int dtype, int64_t T,
                         int64_t E, int64_t k, int score, int renorm, void* dlogits, void* stream) {
  MLP_TRY(check_router(dtype, T, E, k, score, renorm));
  MLP_TRY(need_buf(logits, T, "logits"));
  MLP_TRY(need_buf(ids, T, "ids", false));
  MLP_TRY(need_buf(dweights, T, "dweights", false));
  MLP_TRY(need_buf(dlogits, T, "dlogits"));
  if (T == 0) return MLP_OK;
  return hip_status(run_moe_route_bwd(dtype_of(dtype), logits, ids, dweights, T, (int)E, (int)k, score == MOE_SIGMOID,
                                      renorm, dlogits, stream_of(stream)), "moe_route_bwd");
}

size_t moe_balance_workspace_bytes(int64_t T, int64_t E) {
  if (check_choices(T, E, 1) != MLP_OK) return 0;
  return std::max(kAlign, round_up((size_t)moe_balance_parts(T, (int)E) * (2 * E + 1) * sizeof(float)));
}

mlp_status moe_balance(const void* logits, const int32_t* ids, const uint8_t* mask, int dtype, int64_t T, int64_t E,
                       int64_t k, int score, int32_t* counts, float* shares, float* loss, void* ws, size_t ws_bytes,
                       void* stream) {
  MLP_TRY(check_router(dtype, T, E, k, score, 0));
  MLP_TRY(need_buf(logits, T, "logits"));
  MLP_TRY(need_buf(ids, T, "ids", false));
  MLP_TRY(need_ptr(counts, "counts", false));
  MLP_TRY(need_ptr(shares, "shares", false));
  MLP_TRY(need_ptr(loss, "loss", false));
  const size_t need = moe_balance_workspace_bytes(T, E);
  if (ws_bytes < need)
    return fail(MLP_ERR_WORKSPACE, "workspace of %zu bytes is smaller than the %zu needed", ws_bytes, need);
  MLP_TRY(need_ptr(ws, "workspace"));
  return hip_status(run_moe_balance(dtype_of(dtype), logits, ids, mask, T, (int)E, (int)k, score == MOE_SIGMOID, counts,
                                    shares, loss, ws, stream_of(stream)), "moe_balance");
}

mlp_status moe_balance_bwd(const void* logits, const int32_t* ids, const uint8_t* mask, const int32_t* counts,
                           const float* dloss, const float* dweights, int dtype, int64_t T, int64_t E, int64_t k,
                           int score, int renorm, void* dlogits, void* stream) {
  MLP_TRY(check_router(dtype, T, E, k, score, renorm));
  MLP_TRY(need_buf(logits, T, "logits"));
  if (dweights) MLP_TRY(need_buf(ids, T, "ids", false));
  MLP_TRY(need_ptr(counts, "counts", false));
  if (dloss) MLP_TRY(need_ptr(dloss, "dloss", false));
  if (dweights) MLP_TRY(need_ptr(dweights, "dweights", false));
  MLP_TRY(need_buf(dlogits, T, "dlogits"));
  if (T == 0) return MLP_OK;
  return hip_status(run_moe_balance_bwd(dtype_of(dtype), logits, ids, mask, counts, dloss, dweights, T, (int)E, (int)k,
                                        score == MOE_SIGMOID, renorm, dlogits, stream_of(stream)), "moe_balance_bwd");
}

static mlp_status check_sort(int64_t n, int64_t E) {
  MLP_TRY(check_experts(E));
  if (n < 0) return fail(MLP_ERR_INVALID_ARG, "n = %lld slots", (long long)n);
  if (n > kRowLimit) return fail(MLP_ERR_UNSUPPORTED, "n is above 2^30");
  return MLP_OK;
}

size_t moe_sort_workspace_bytes(int64_t n, int64_t E) {
  if (check_sort(n, E) != MLP_OK) return 0;
  return std::max(kAlign, round_up(moe_sort_counts_bytes(n, (int)E)));
}

mlp_status moe_sort(const int32_t* ids, int64_t n, int64_t E, int32_t* offsets, int32_t* row_of, int32_t* slot_of,
                    void* ws, size_t ws_bytes, void* stream) {
  MLP_TRY(check_sort(n, E));
  MLP_TRY(need_buf(ids, n, "ids", false));
  MLP_TRY(need_ptr(offsets, "offsets", false));
  MLP_TRY(need_buf(row_of, n, "row_of", false));
  MLP_TRY(need_buf(slot_of, n, "slot_of", false));
  const size_t need = moe_sort_workspace_bytes(n, E);
  if (ws_bytes < need)
    return fail(MLP_ERR_WORKSPACE, "workspace of %zu bytes is smaller than the %zu needed", ws_bytes, need);
  MLP_TRY(need_ptr(ws, "workspace"));
  return hip_status(run_moe_sort(ids, n, (int)E, offsets, row_of, slot_of, static_cast<int*>(ws), stream_of(stream)),
                    "moe_sort");
}

mlp_status moe_gather(const void* x, const int32_t* slot_of, const int32_t* offsets, int dtype, int64_t T, int64_t E,
                      int64_t k, int64_t d, void* xs, void* stream) {
  MLP_TRY(check_rows(dtype, T, E, k, d));
  MLP_TRY(need_buf(x, T, "x"));
  MLP_TRY(need_buf(slot_of, T, "slot_of", false));
  MLP_TRY(need_ptr(offsets, "offsets", false));
  MLP_TRY(need_buf(xs, T, "xs"));
  if (T == 0) return MLP_OK;
  return hip_status(run_moe_gather(x, slot_of, offsets, (int)(T * k), (int)E, (int)k, pieces_of(dtype, d), xs,
                                   stream_of(stream)), "moe_gather");
}

mlp_status moe_gather_bwd(const void* dxs, const int32_t* row_of, const int32_t* offsets, int dtype, int64_t T,
                          int64_t E, int64_t k, int64_t d, void* dx, void* stream) {
  MLP_TRY(check_rows(dtype, T, E, k, d));
  MLP_TRY(need_buf(dxs, T, "dxs"));
  MLP_TRY(need_buf(row_of, T, "row_of", false));
  MLP_TRY(need_ptr(offsets, "offsets", false));
  MLP_TRY(need_buf(dx, T, "dx"));
  if (T == 0) return MLP_OK;
  return hip_status(run_moe_combine(dtype_of(dtype), dxs, nullptr, row_of, offsets, nullptr, (int)T, (int)E, (int)k,
                                    pieces_of(dtype, d), dx, stream_of(stream)), "moe_gather_bwd");
}

mlp_status moe_combine(const void* ys, const float* weights, const int32_t* row_of, const int32_t* offsets,
                       const void* residual, int dtype, int64_t T, int64_t E, int64_t k, int64_t d, void* out,
                       void* stream) {
  MLP_TRY(check_rows(dtype, T, E, k, d));
  MLP_TRY(need_buf(ys, T, "ys"));
  MLP_TRY(need_buf(weights, T, "weights", false));
  MLP_TRY(need_buf(row_of, T, "row_of", false));
  MLP_TRY(need_ptr(offsets, "offsets", false));
  if (residual) MLP_TRY(need_ptr(residual, "residual"));
  MLP_TRY(need_buf(out, T, "out"));
  if (T == 0) return MLP_OK;
  return hip_status(run_moe_combine(dtype_of(dtype), ys, weights, row_of, offsets, residual, (int)T, (int)E, (int)k,
                                    pieces_of(dtype, d), out, stream_of(stream)), "moe_combine");
}

mlp_status moe_combine_bwd(const void* dout, const void* ys, const float* weights, const int32_t* slot_of,
                           const int32_t* offsets, int dtype, int64_t T, int64_t E, int64_t k, int64_t d, void* dys,
                           float* dweights, void* stream) {
  MLP_TRY(check_rows(dtype, T, E, k, d));
  MLP_TRY(need_buf(dout, T, "dout"));
  MLP_TRY(need_buf(ys, T, "ys"));
  MLP_TRY(need_buf(weights, T, "weights", false));
  MLP_TRY(need_buf(slot_of, T, "slot_of", false));
  MLP_TRY(need_ptr(offsets, "offsets", false));
  MLP_TRY(need_buf(dys, T, "dys"));
  MLP_TRY(need_buf(dweights, T, "dweights", false));
  if (T == 0) return MLP_OK;
  return hip_status(run_moe_combine_bwd(dtype_of(dtype), dout, ys, weights, slot_of, offsets, (int)(T * k),
                                        (int)E, (int)k, pieces_of(dtype, d), dys, dweights, stream_of(stream)),
                    "moe_combine_bwd");
}

size_t linear_workspace_bytes(const linear_desc* d, int phase) {
  if (check_linear(d) != MLP_OK) return 0;
  if (phase != LINEAR_FWD && phase != LINEAR_BWD) {
    fail(MLP_ERR_INVALID_ARG, "phase %d is not a linear_phase", phase);
    return 0;
  }
  return linear_ws(d, phase).total;
}

mlp_status linear_fwd(const linear_desc* d, const void* x, const void* w, const void* w_up, const void* bias,
                      const void* bias_up, const void* residual, const int32_t* offsets, void* y, void* preact,
                      void* ws, size_t ws_bytes, void* stream) {
  MLP_TRY(check_linear(d));
  const bool gated = is_gated(d->act);
  MLP_TRY(check_weights(d, x, w, w_up, offsets));
  if (bias) MLP_TRY(need_ptr(bias, "bias"));
  if (gated && (bias == nullptr) != (bias_up == nullptr))
    return fail(MLP_ERR_INVALID_ARG, "bias and bias_up must both be given or both be NULL");
  if (!gated) MLP_TRY(need_null(bias_up, "bias_up", "unless the activation is gated"));
  if (bias_up) MLP_TRY(need_ptr(bias_up, "bias_up"));
  if (residual) MLP_TRY(need_ptr(residual, "residual"));
  MLP_TRY(need_buf(y, d->M, "y"));
  if (preact) MLP_TRY(need_ptr(preact, "preact"));
  MLP_TRY(check_linear_ws(d, LINEAR_FWD, ws, ws_bytes));
  if (d->M == 0) return MLP_OK;

  hipStream_t s = stream_of(stream);
  const DType io = dtype_of(d->dtype);
  const int64_t M = d->M, N = d->N, K = d->K, P = gated ? 2 * N : N;
  const int epi = gated ? EPI_LIN_GATED : EPI_LIN;
  GemmArgs a = linear_args(d);
  a.A = x;
  a.lda = a.ldb = K;
  a.B0 = w;
  a.B1 = w_up;
  a.C0 = y;
  a.ldc0 = N;
  a.aux = preact;
  a.ld_aux = P;
  a.half = (int)N;
  a.flags = preact ? 1 : 0;
  a.bias0 = bias;
  a.bias1 = bias_up;
  a.res = residual;
  a.ld_res = N;

  if (d->experts) {
    const ExpertPlan p = plan_experts(d, true);
    a.N = (int)N;
    a.K = a.k_per_split = (int)K;
    ExpertGemm e = expert_gemm(d, a, offsets);
    if (p.form == EXPERT_SKINNY) {
      e.grid = (int)(d->experts + 1 + (M - 1) / 16);   // runs of column blocks
      return hip_status(run_skinny_experts(io, epi, e, s), "experts' products (few rows)");
    }
    const int64_t bn = gated ? p.bn / 2 : p.bn;
    e.g.tiles_n = (int)((N + bn - 1) / bn);
    e.g.group_m = 8;
    e.grid = (int)(row_tiles(M, d->experts, p.bm) * e.g.tiles_n);
    if (p.tile == TILE_256x256_W8) {
      e.split_tail = 1;
      e.grid += 128;   // the tail's second halves
    }
    return hip_status(run_expert_fwd(io, epi, p.tile, e, s), "experts' products");
  }
  const LinearFwd f = plan_linear(d);
  if (f.skinny) return hip_status(run_skinny(io, epi, planned(a, Plan{}, M, N, K), s), "linear layer (small M)");
  if (f.plan.splits > 1) {
    GemmArgs b = planned(a, f.plan, M, P, K);
    if (gated) b.b_split = (int)N;   // [w; w_up] stacked along the output columns
    b.partial = static_cast<float*>(ws);
    MLP_TRY(hip_status(run_gemm(io, DT_F32, NT, EPI_PARTIAL, f.plan.tile, b, f.plan.grid, s), "linear layer (partial sums)"));
    return hip_status(run_linear_reduce(io, gated, b.partial, f.plan.splits, planned(a, f.plan, M, N, K), s),
                      "linear layer (join)");
  }
  return hip_status(run_gemm_linear(io, epi, f.plan.tile, planned(a, f.plan, M, N, K), f.plan.grid, s), "linear layer");
}

mlp_status linear_bwd(const linear_desc* d, const void* dy, const void* x, const void* w, const void* w_up,
                      const void* preact, const int32_t* offsets, void* dx, void* dw, void* dw_up, void* dbias,
                      void* dbias_up, int grad_accum, void* ws, size_t ws_bytes, void* stream) {
  MLP_TRY(check_linear(d));
  const bool gated = is_gated(d->act), act = d->act != LINEAR_ACT_NONE;
  MLP_TRY(need_buf(dy, d->M, "dy"));
  MLP_TRY(check_weights(d, x, w, w_up, offsets));
  if (act) MLP_TRY(need_buf(preact, d->M, "preact"));
  else MLP_TRY(need_null(preact, "preact", "without an activation"));
  if (dx) MLP_TRY(need_ptr(dx, "dx"));
  if (gated) {
    if ((dw == nullptr) != (dw_up == nullptr))
      return fail(MLP_ERR_INVALID_ARG, "dw and dw_up must both be given or both be NULL");
    if ((dbias == nullptr) != (dbias_up == nullptr))
      return fail(MLP_ERR_INVALID_ARG, "dbias and dbias_up must both be given or both be NULL");
  } else {
    MLP_TRY(need_null(dw_up, "dw_up", "unless the activation is gated"));
    MLP_TRY(need_null(dbias_up, "dbias_up", "unless the activation is gated"));
  }
  if (dw) MLP_TRY(need_ptr(dw, "dw"));
  if (dw_up) MLP_TRY(need_ptr(dw_up, "dw_up"));
  if (dbias) MLP_TRY(need_ptr(dbias, "dbias"));
  if (dbias_up) MLP_TRY(need_ptr(dbias_up, "dbias_up"));
  if (grad_accum != 0 && grad_accum != 1) return fail(MLP_ERR_INVALID_ARG, "grad_accum must be 0 or 1");
  MLP_TRY(check_linear_ws(d, LINEAR_BWD, ws, ws_bytes));

  hipStream_t s = stream_of(stream);
  const DType io = dtype_of(d->dtype), gio = grad_accum ? DT_F32 : io;
  const int64_t M = d->M, N = d->N, K = d->K, P = gated ? 2 * N : N, E = std::max(d->experts, 1);
  const LinearWs L = linear_ws(d, LINEAR_BWD);
  char* base = static_cast<char*>(ws);
  const bool need_dz = act && (dx || dw) && M > 0;
  float* sums = reinterpret_cast<float*>(base + L.sums);
  void* dz = need_dz ? base + L.dz : nullptr;
  if ((need_dz || dbias) && M > 0)
    MLP_TRY(hip_status(run_linear_dact(io, gated, linear_args(d).act, dy, preact, offsets, (int)E, M, N, dz,
                                       dbias ? sums : nullptr, s), "activation gradient"));
  BiasGrad db{};
  if (dbias) {
    db = {sums, offsets, (int)E, (int)M, (int)N, dact_rows(M, N), (int)dact_pieces(M, N, E), grad_accum, dbias, dbias_up, 0, 1};
    const int64_t pieces = M / E / dact_rows(M, N);   // of an expert
    db.runs = pieces <= 16 ? 1 : pieces <= 64 ? 4 : 16;
    db.grid = (int)(E * ((P + 256 / db.runs - 1) / (256 / db.runs)));
  }
  const LinearBwd b = d->experts || M == 0 ? LinearBwd{} : plan_linear_bwd(d, dx != nullptr, dw != nullptr);
  const bool one = d->experts || M == 0 || b.small;   // (one weight without rows: as one expert without rows)
  if (dbias && (!one || (!dx && !dw))) MLP_TRY(hip_status(run_linear_dbias(io, db, s), "bias gradient"));
  if (!dx && !dw) return MLP_OK;

  GemmArgs gx = linear_args(d);   // dx = dz [W; W_up]
  gx.A = act ? dz : dy;
  gx.lda = P;
  gx.B0 = w;
  gx.B1 = w_up;
  if (gated) gx.b_split = (int)N;
  gx.ldb = K;
  gx.C0 = dx;
  gx.ldc0 = K;
  GemmArgs gw = linear_args(d);   // [dW; dW_up] = dz^T x
  gw.A = gx.A;
  gw.lda = P;
  gw.B0 = x;
  gw.ldb = K;
  gw.C0 = dw;
  gw.C1 = dw_up;
  if (gated) gw.c_split = (int)N;
  gw.ldc0 = K;
  gw.accumulate = grad_accum;

  if (one) {
    const ExpertPlan p = plan_experts(d, false);
    ExpertBwd b{};
    b.db = db;
    gx.N = (int)K;
    gx.K = gx.k_per_split = (int)P;
    gx.tiles_n = (int)((K + p.bn - 1) / p.bn);
    gx.group_m = 8;
    b.dx = expert_gemm(d, gx, offsets);
    b.dx_splits = dx ? p.dx_splits : 1;
    b.dx_kps = b.dx_splits > 1 ? (int)((P + b.dx_splits - 1) / b.dx_splits + bk_of(io) - 1) / bk_of(io) * bk_of(io) : (int)P;
    if (b.dx_splits > 1) b.dx_splits = (int)((P + b.dx_kps - 1) / b.dx_kps);
    b.part_x = reinterpret_cast<float*>(base + L.partial);
    if (dx && M > 0) b.dx.grid = (int)((row_tiles(M, E, p.bm) * gx.tiles_n * b.dx_splits + 7) / 8 * 8);
    gw.M = (int)P;
    gw.N = (int)K;
    gw.tiles_m = (int)((P + p.bm - 1) / p.bm);
    gw.tiles_n = (int)((K + p.bn - 1) / p.bn);
    gw.group_m = std::min(gw.tiles_m, 8);
    if (p.strip_parts) {
      gw.tiles_m = (int)((P + kStripTileM - 1) / kStripTileM);
      gw.tiles_n = (int)((K + kStripTileN - 1) / kStripTileN);
      b.strip_parts = p.strip_parts;
    }
    if (E * P * K * esize(d->dtype) >= kStreamGradBytes)
      gw.flags = kFlagLarge | (!p.strip_parts || K * esize(d->dtype) % 128 == 0 ? kFlagStream : 0);
    b.dw = expert_gemm(d, gw, offsets);
    if (dw && M > 0) {
      b.piece_rows = p.piece_rows;
      b.max_slots = p.max_slots;
      b.part_w = reinterpret_cast<float*>(base + L.part_w);
    }
    const int64_t shares = (int64_t)(b.strip_parts ? b.strip_parts : gw.tiles_m) * gw.tiles_n;   // of an expert's weight gradient
    if (dw) b.dw.grid = (int)(((b.piece_rows ? M / b.piece_rows : 0) + E) * shares);
    if (dw && b.dx.grid && p.dw_first) {
      b.dw_first = 1;
      if (b.piece_rows) b.dw.grid = (b.dw.grid + 7) / 8 * 8;
    }
    if (b.dx.grid + b.dw.grid + b.db.grid == 0) return MLP_OK;
    MLP_TRY(hip_status(run_expert_bwd(io, p.tile, b, s), "experts' gradients"));
    return hip_status(run_expert_join(io, b, s), "experts' gradients (join)");
  }
  void* partial = base + L.partial;
  if (b.group) {
    GemmGroup g{};
    const bool dx_first = P >= M;   // longest K first
    const Plan* plans[2] = {dx_first ? &b.gdx : &b.gdw, dx_first ? &b.gdw : &b.gdx};
    g.g[dx_first ? 0 : 1] = planned(gx, b.gdx, M, K, P);
    g.g[dx_first ? 1 : 0] = planned(gw, b.gdw, P, K, M);
    for (int j = 0; j < 2; ++j) {
      g.kind[j] = (j == 0) == dx_first ? 0 : 1;
      g.items[j] = plans[j]->grid;
      g.begin[j + 1] = g.begin[j] + (plans[j]->grid + 7) / 8 * 8;
    }
    g.count = 2;
    return hip_status(run_gemm_group16(io, gio, EPI_STORE, g, s), "linear layer's gradients (one launch)");
  }
  if (dx) MLP_TRY(gemm_rows(io, io, NN, b.dx, gx, M, K, P, partial, s, "linear layer's dx"));
  if (dw) MLP_TRY(gemm(io, gio, TN, EPI_STORE, b.dw, gw, P, K, M, partial, s, "linear layer's dW"));
  return MLP_OK;
}

}  // extern "C"

namespace gmlp {

hipError_t run_gemm_linear(DType in, int epi, TileShape tile, const GemmArgs& a, int grid, hipStream_t s) {
  if (tile == TILE_64x64 && in != DT_F32) return run_gemm_small16(in, in, NT, epi, a, grid, s);
  switch (in) {
    case DT_BF16: return run_gemm_bf16_linear(epi, tile, a, grid, s);
    case DT_F16: return run_gemm_f16_linear(epi, tile, a, grid, s);
    case DT_F32: return run_gemm_f32_ring(NT, epi, tile, a, grid, s);
    default: return hipErrorInvalidValue;
  }
}

hipError_t run_expert_fwd(DType in, int epi, TileShape tile, const ExpertGemm& a, hipStream_t s) {
  switch (in) {
    case DT_BF16: return run_expert_fwd_bf16(epi, tile, a, s);
    case DT_F16: return run_expert_fwd_f16(epi, tile, a, s);
    case DT_F32: return run_expert_fwd_f32(epi, tile, a, s);
    default: return hipErrorInvalidValue;
  }
}

hipError_t run_expert_bwd(DType in, TileShape tile, const ExpertBwd& a, hipStream_t s) {
  switch (in) {
    case DT_BF16: return run_expert_bwd_bf16(tile, a, s);
    case DT_F16: return run_expert_bwd_f16(tile, a, s);
    case DT_F32: return run_expert_bwd_f32(tile, a, s);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace gmlp
