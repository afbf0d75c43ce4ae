// Host-side pieces the C-ABI translation units share: error text, argument checks, the GEMM
// planner and planned launches. Defined in mlp_api.hip unless inline here.
#pragma once

#include <stddef.h>
#include <stdint.h>

#include "launch.hpp"
#include "mlp.h"

namespace gmlp {

// Records the text mlp_last_error() returns on this thread and hands `st` back.
mlp_status fail(mlp_status st, const char* fmt, ...);
mlp_status hip_status(hipError_t e, const char* what);
mlp_status need_ptr(const void* p, const char* name, bool align = true);   // non-NULL, 16- (else 4-) byte aligned
mlp_status need_null(const void* p, const char* name, const char* why);

#define MLP_TRY(expr)                 \
  do {                                \
    const mlp_status st_ = (expr);    \
    if (st_ != MLP_OK) return st_;    \
  } while (0)

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

constexpr size_t kAlign = 256;
inline size_t round_up(size_t v) { return (v + kAlign - 1) / kAlign * kAlign; }

inline int esize(int dtype) { return dtype == MLP_F32 ? 4 : 2; }

inline bool is_gated(int act) {
  return act == MLP_ACT_SWIGLU || act == MLP_ACT_GEGLU || act == MLP_ACT_REGLU || act == MLP_ACT_GLU;
}

// The epilogues' function of an mlp_act: the gate function of a gated one, else f itself.
inline int act_fn_of(int act) {
  switch (act) {
    case MLP_ACT_SWIGLU: return FN_SILU;
    case MLP_ACT_GEGLU: case MLP_ACT_GELU_TANH: return FN_GELU_TANH;
    case MLP_ACT_REGLU: case MLP_ACT_RELU: return FN_RELU;
    case MLP_ACT_GLU: return FN_SIGMOID;
    default: return FN_RELU_SQ;
  }
}
inline DType dtype_of(int dtype) { return dtype == MLP_BF16 ? DT_BF16 : dtype == MLP_F16 ? DT_F16 : DT_F32; }

// ---- GEMM planning ---------------------------------------------------------------------------

struct Plan {
  TileShape tile;
  int splits, k_per_split, tiles_m, tiles_n, group_m, grid;
  double est;   // the planner's time model of this plan, seconds
};

struct TileInfo { TileShape t; int bm, bn, slots; double eff; };
constexpr int kTileInfos = 5;
extern const TileInfo kTiles[kTileInfos];

inline bool is_fp8(DType in) { return in == DT_E4M3 || in == DT_F8G; }
int bk_of(DType in);   // K elements of one K-step

// gated: N counts hidden units and a tile covers bn/2 of them (gate + up rows). only_tile >= 0
// restricts the choice to that tile shape.
Plan plan_gemm(DType in, int64_t M, int64_t N, int64_t K, bool allow_split, bool gated, int only_tile = -1);
// The same over another list of tile shapes.
Plan plan_tiles(const TileInfo* tiles, int count, DType in, int64_t M, int64_t N, int64_t K, bool allow_split,
                bool gated);
size_t partial_bytes(const Plan& p, int64_t M, int64_t N);

// A store-epilogue GEMM cut along M: rows [0, m1) by `main`, the rest by `tail` (m1 = 0: all by
// `main`); see plan_rows.
struct RowsPlan {
  Plan main{};
  int64_t m1 = 0;
  Plan tail{};
};
RowsPlan plan_rows(DType in, int64_t M, int64_t N, int64_t K);
size_t partial_bytes(const RowsPlan& r, int64_t M, int64_t N);

double list_makespan(const int64_t* tiles, const int64_t* steps, int count, double overhead);

// ---- planned launches --------------------------------------------------------------------------

GemmArgs planned(GemmArgs a, const Plan& p, int64_t M, int64_t N, int64_t K);
mlp_status gemm(DType in, DType io, Layout lay, int epi, const Plan& p, GemmArgs a, int64_t M, int64_t N, int64_t K,
                void* partial, hipStream_t s, const char* what);
mlp_status gemm_rows(DType in, DType io, Layout lay, const RowsPlan& r, GemmArgs a, int64_t M, int64_t N, int64_t K,
                     void* partial, hipStream_t s, const char* what);

}  // namespace gmlp
