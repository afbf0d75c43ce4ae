// Arguments of the MLP engine's GEMM kernel, shared by host dispatch and device code.
#pragma once

#include <stdint.h>

namespace gmlp {

// The activation functions of the fused epilogues (GemmArgs::act): the gate function f of a
// gated activation a = f(g) * u (SwiGLU: silu, GeGLU: gelu_tanh, ReGLU: relu, GLU: sigmoid), or
// the f of a non-gated post = f(pre) (relu^2, relu, gelu_tanh).
// FN_NONE: the linear epilogues only.
enum ActFn : int { FN_SILU = 0, FN_GELU_TANH = 1, FN_RELU = 2, FN_SIGMOID = 3, FN_RELU_SQ = 4, FN_NONE = 5 };

enum Epi : int {
  EPI_STORE = 0,    // C = alpha * acc (OutT); accumulate: C(f32) += alpha * acc; rows >= c_split go to C1
  EPI_PARTIAL = 1,  // split-K: partial[split][m][n] = acc (fp32); a reduce kernel finishes
  EPI_GATED = 2,    // g, u = alpha * acc pair; aux[m][n], aux[m][half+n] = g, u (flag 1);
                    // C0[m][n] = a = act(g, u) (flag 2), act per GemmArgs::act
  EPI_ACT = 3,      // pre = alpha * acc -> aux (flag 1); post = f(pre) -> C0 (flag 2)
  EPI_DGATED = 4,   // da = alpha * acc; g, u <- aux; dg, du -> C0[m][n], C0[m][half+n];
                    // a -> C1 (flag 2). C0 may equal aux.
  EPI_DACT = 5,     // dpost = alpha * acc; pre <- aux; dpre = dpost * f'(pre) -> C0; post -> C1 (flag 2)
  EPI_F8ACT = 6,    // pre = alpha * acc -> aux (bf16 or fp32, flag 1); post = relu(pre)^2;
                    // C0 = e4m3(post / *s_post); *amax = max(*amax, max post)
  EPI_F8DACT = 7,   // dpre = alpha * acc * 2 max(pre, 0), pre <- aux (bf16 or fp32);
                    // C0 = e5m2(dpre / *s_post) (s_post holds the dpre scale here);
                    // *amax = max(*amax, max |dpre|); C1 set: C1 = e4m3(relu(pre)^2 / *s_c1)
  EPI_LIN = 8,      // z = acc + bias0[n] -> aux (flag 1); C0 = res + f(z) (bias0, res may be NULL)
  EPI_LIN_GATED = 9,// g, u = acc pair + bias0[n], bias1[n] -> aux[m][n], aux[m][half+n] (flag 1);
                    // C0 = res + f(g) u
  EPI_STORE_PART = 10   // STORE, or with partial set the accumulators in fp32 to partial[m][n]
};

// Epilogues whose tile holds gate rows and the up rows of the same units.
constexpr bool epi_gated(int epi) { return epi == EPI_GATED || epi == EPI_LIN_GATED; }
constexpr bool epi_linear(int epi) { return epi == EPI_LIN || epi == EPI_LIN_GATED; }

struct GemmArgs {
  int M, N, K;
  const void* A; int64_t lda;
  // B from two matrices when B1 is set: MN-major B stacked along K (rows k >= b_split from B1,
  // the [W_gate; W_up] of dx); K-major non-gated B stacked along N (rows n >= b_split from B1)
  const void* B0; const void* B1; int64_t ldb; int b_split;
  void* C0; int64_t ldc0; void* C1; int64_t ldc1; int c_split;
  void* aux; int64_t ld_aux; int half;
  float alpha; const float* alpha_dev0; const float* alpha_dev1;
  float gate_mult; int gate_inside;
  int act;          // ActFn of the GATED / DGATED / ACT / DACT epilogues (F8ACT is relu^2)
  int accumulate;
  int flags;
  const float* s_post; float* amax;
  int k_per_split; float* partial;
  int tiles_m, tiles_n, group_m;
  const float* s_c1;   // F8DACT: scale of the e4m3 relu(pre)^2 codes written to C1
  const void* bias0; const void* bias1; const void* res; int64_t ld_res;   // LIN, LIN_GATED
};

// One product an expert, rows grouped by expert: expert e has rows offsets[e] .. offsets[e+1]-1 of
// the row-indexed operands (offsets NULL: one expert with all rows) and weight matrices, biases and
// weight gradients w_stride, bias_stride and w_stride elements apart. The members' pointers are those
// of expert 0 and row 0; M (products over rows) or K (weight gradients) is set per expert on the
// device. tiles_m of a product over rows is unused.
// In g.flags: an output that no cache holds until it is read is stored past the caches; so are its runs of zeros.
constexpr int kFlagStream = 4, kFlagLarge = 8;
struct ExpertGemm {
  GemmArgs g;
  const int* offsets;
  int experts, rows;
  int64_t w_stride, bias_stride;
  int grid;   // workgroups: an upper bound of the tiles for a product over rows
  int split_tail;   // products over rows in 256-row tiles: a last round of at most half the CUs runs as halves
};
// The bias gradients from the column sums of pieces of at most `step` rows (run_linear_dact): db0
// [experts, N], and db1 for the other N columns of a gated layer; written, or added into fp32. runs (1, 4, 16): parts of
// an expert's pieces that are summed beside one another.
struct BiasGrad {
  const float* sums;
  const int* offsets;
  int experts, rows, N, step, max_pieces, accumulate;
  void* db0; void* db1;
  int grid, runs;
};
// The backward's two products and the bias gradient in one launch: the workgroups of dx and of dW (dw_first:
// the other way round), then the bias gradient's.
//  * dx_splits > 1: dx's K in parts of dx_kps, fp32 sums in part_x [dx_splits][rows][N];
//  * piece_rows: an expert of more rows has its weight gradient summed over pieces of that many, fp32 sums in
//    part_w [slots][M][N], slots counted over such experts in order, max_slots at most (0: never).
// run_expert_join adds up either.
//  * strip_parts > 0: few rows an expert. dx in 64 x 128 tiles; the weight gradients 128 columns of x a workgroup
//    (kStripTileN), every strip_parts-th of the 64-column tiles of dz (kStripTileM) one after another (expert_grad_strip).
struct ExpertBwd {
  ExpertGemm dx, dw;
  BiasGrad db;
  int dw_first;
  int dx_splits, dx_kps; float* part_x;
  int piece_rows, max_slots; float* part_w;
  int strip_parts;
};

// Up to kGroupMax independent GEMMs run by one launch (gemm_dma_group_kernel): member j covers
// workgroups [begin[j], begin[j+1]) (multiples of 8 apart), has items[j] tiles (one per
// workgroup, no split) and takes tile body kind[j] (0 or 1) of the kernel's two.
constexpr int kGroupMax = 3;
struct GemmGroup {
  GemmArgs g[kGroupMax];
  int begin[kGroupMax + 1];
  int items[kGroupMax];
  int kind[kGroupMax];
  int count;
};

}  // namespace gmlp
