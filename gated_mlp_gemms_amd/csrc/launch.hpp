// Host-side declarations of every kernel launch the C-ABI layer uses.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "gemm_args.hpp"

namespace gmlp {

// DT_F8G: the fp8-gradient GEMM operand pair (A e5m2, B e4m3); an input type only.
enum DType : int { DT_F32 = 0, DT_BF16 = 1, DT_E4M3 = 2, DT_F16 = 3, DT_F8G = 4 };
enum Layout : int { NT = 0, NN = 1, TN = 2 };   // A K-major/B K-major, A K/B MN, A MN/B MN
// Tile shapes of the bf16 / e4m3 kernel; _W8 runs the tile with 8 waves (two per SIMD). _RING: the
// linear layer's and the experts' fp32 tile on the 16-bit kernels' DMA ring; TILE_64x64: theirs for small
// products, every type (64 x 128 where a tile holds gate and up rows).
enum TileShape : int {
  TILE_256x256 = 0, TILE_256x128 = 1, TILE_128x128 = 2, TILE_256x256_W8 = 3, TILE_256x128_W8 = 4, TILE_128x128_RING = 5,
  TILE_64x64 = 6, TILE_COUNT = 7
};

// One GEMM launch. `io` is the element type of the epilogue's stored/loaded tensors (for
// EPI_STORE the output type; accumulate mode needs DT_F32). Returns hipErrorInvalidValue for a
// combination that has no instantiation.
hipError_t run_gemm(DType in, DType io, Layout layout, int epi, TileShape tile, const GemmArgs& a,
                    int grid, hipStream_t stream);

// Per-(input dtype, layout) launchers, one translation unit each.
hipError_t run_gemm_bf16_nt(DType io, int epi, TileShape tile, const GemmArgs& a, int grid, hipStream_t s);
hipError_t run_gemm_bf16_nn(DType io, int epi, TileShape tile, const GemmArgs& a, int grid, hipStream_t s);
hipError_t run_gemm_bf16_tn(DType io, int epi, TileShape tile, const GemmArgs& a, int grid, hipStream_t s);
hipError_t run_gemm_f16_nt(DType io, int epi, TileShape tile, const GemmArgs& a, int grid, hipStream_t s);
hipError_t run_gemm_f16_nn(DType io, int epi, TileShape tile, const GemmArgs& a, int grid, hipStream_t s);
hipError_t run_gemm_f16_tn(DType io, int epi, TileShape tile, const GemmArgs& a, int grid, hipStream_t s);
hipError_t run_gemm_f32(Layout layout, int epi, TileShape tile, const GemmArgs& a, int grid, hipStream_t s);
hipError_t run_gemm_e4m3_nt(DType io, int epi, TileShape tile, const GemmArgs& a, int grid, hipStream_t s);
hipError_t run_gemm_f8g_nt(DType io, int epi, TileShape tile, const GemmArgs& a, int grid, hipStream_t s);
hipError_t run_gemm_f8g_tn(DType io, int epi, TileShape tile, const GemmArgs& a, int grid, hipStream_t s);

// Independent GEMMs of the 16-bit backward in one launch of 8-wave 256 x 256 tiles (GemmGroup):
// kind 0 an NN product with epilogue epi0 (EPI_STORE: dx; EPI_DGATED / EPI_DACT: the
// d-activation GEMM), output `in`; kind 1 a TN weight gradient with the store epilogue, output
// gio (`in`, or DT_F32 to accumulate).
hipError_t run_gemm_group16(DType in, DType gio, int epi0, const GemmGroup& g, hipStream_t s);

// Products with at most kSkinnyMaxRows rows (decode-size token counts), K-major A [M, K] and
// B [N, K] (gated: B0 gate rows, B1 up rows), in `in` = DT_BF16 / DT_F16; K a multiple of 8.
// Epilogues EPI_STORE (C0 = alpha * A B^T), EPI_ACT and EPI_GATED with GemmArgs::flags as in the
// GEMM kernels (bit 0: the pre-activation into aux, bit 1: the activation into C0).
constexpr int kSkinnyMaxRows = 16;
hipError_t run_skinny(DType in, int epi, const GemmArgs& a, hipStream_t s);
// EPI_PARTIAL: the store product with K split over kSkinnyParts workgroups per column block,
// unscaled fp32 partial sums into a.partial [kSkinnyParts][M][N] (then the split-K reduce).
// Taken above 8 tokens for narrow outputs with a long K (skinny_parts_for), where the whole-K
// form has few column blocks and each of them re-reads all of the token rows. LLaMA widths, same
// box: 16 tokens 60.8 -> 57.5 us per inference forward; 8 and 1 tokens 54.3 -> 56.4 and 48.6 ->
// 53.1 us (few token rows to save, one more launch), hence the threshold.
constexpr int kSkinnyParts = 4;
inline bool skinny_parts_for(int64_t M, int64_t N, int64_t K) { return M > 8 && N <= 8192 && K >= 2048; }

// ---- linear layer and the experts' products ----------------------------------------------------

// y = res + act(x W^T + b): EPI_LIN or EPI_LIN_GATED, K-major operands in `in`, unsplit.
hipError_t run_gemm_linear(DType in, int epi, TileShape tile, const GemmArgs& a, int grid, hipStream_t s);
hipError_t run_gemm_bf16_linear(int epi, TileShape tile, const GemmArgs& a, int grid, hipStream_t s);
hipError_t run_gemm_f16_linear(int epi, TileShape tile, const GemmArgs& a, int grid, hipStream_t s);
// 16-bit 64 x 64 tiles, the same products.
hipError_t run_gemm_small16(DType in, DType io, Layout layout, int epi, const GemmArgs& a, int grid, hipStream_t s);
// fp32 on the DMA ring: NT with the linear epilogues or partial sums, NN and TN with the store or those.
hipError_t run_gemm_f32_ring(Layout layout, int epi, TileShape tile, const GemmArgs& a, int grid, hipStream_t s);
// The same from fp32 partials [splits][M][N] (gated: [splits][M][2N], g then u), summed in order.
hipError_t run_linear_reduce(DType io, int gated, const float* partial, int splits, const GemmArgs& a, hipStream_t s);

// One product an expert (ExpertGemm). Tiles: TILE_256x256_W8, TILE_128x128 (f32: its _RING) and
// TILE_64x64.
hipError_t run_expert_fwd(DType in, int epi, TileShape tile, const ExpertGemm& a, hipStream_t s);
hipError_t run_expert_bwd(DType in, TileShape tile, const ExpertBwd& a, hipStream_t s);
hipError_t run_expert_fwd_bf16(int epi, TileShape tile, const ExpertGemm& a, hipStream_t s);
hipError_t run_expert_fwd_f16(int epi, TileShape tile, const ExpertGemm& a, hipStream_t s);
hipError_t run_expert_fwd_f32(int epi, TileShape tile, const ExpertGemm& a, hipStream_t s);
hipError_t run_expert_bwd_bf16(TileShape tile, const ExpertBwd& a, hipStream_t s);
hipError_t run_expert_bwd_f16(TileShape tile, const ExpertBwd& a, hipStream_t s);
hipError_t run_expert_bwd_f32(TileShape tile, const ExpertBwd& a, hipStream_t s);
// Few rows an expert (ExpertBwd::strip_parts, 16-bit): weight gradients in tiles of kStripTileM columns of dz by
// kStripTileN of x. Taken up to kStripRows rows an expert on average, for weight gradients that caches hold
// (kStreamGradBytes) up to kStripRowsSmall. Both products, against the tiles (us): 1711 rows of 113 experts (6080 x 152) 147
// and 197, 97 of 60 (4992 x 704) 212 and 243, 4096 of 32 (2048 x 1376) 110 and 95; caches hold: 5 of 3 (4456 x 464) 15 and 23,
// 576 of 3 (1952 x 672) 19 and 23, 4000 of 16 (512 x 1024) 37 and 31.
constexpr int kStripTileM = 64, kStripTileN = 128, kStripRows = 32, kStripRowsSmall = 200;
// Weight gradients from this size on are stored past the caches (16-bit; in strips only with rows of whole 128-byte
// lines: a strip's store of part of a line goes to memory on its own). Both products, into caches and past them (us), 24
// rows an expert of 2048 x 1376 gate and up: gradients of 50 MB 40 and 37, 90 MB 65 and 54, 110 MB 78 and 72, 180 MB 114
// and 106; 400 rows: 50 MB 77 and 69, 110 MB 139 and 137, 180 MB 229 and 225. A reader right after the call would rather
// find them in the caches (24 rows, the gradients scaled by a pass of its own: 50 MB 57 and 58, 90 MB 90 and 95, 110 MB
// 109 and 114, 180 MB 163 and 175); a training step reads them when the other layers' have passed, and the larger they
// are the less of them a cache has kept.
constexpr int64_t kStreamGradBytes = 100 << 20;
// The partial sums of run_expert_bwd added up (nothing without any).
hipError_t run_expert_join(DType io, const ExpertBwd& a, hipStream_t s);
// The forward with a few rows an expert, 16-bit (g.N output columns, any rows; grid: runs of column blocks).
// Taken up to kExpertFewRows rows an expert on average (an expert's weights are streamed again for every 16 of its rows).
// Streamed and in tiles (us, even and uneven rows): at 8 rows an expert, 4 experts of 1024 x 1024 4.4 and 8.7, 32 of 512 x 264
// 5-7 and 7, 8 of 2048 x 5504 gate and up 70-75 and 80, 16 of 4096 x 1408 gate and up 75 and 76, 64 of 1376 x 2048 79 and 73,
// 64 of 2048 x 1376 gate and up 139-149 and 124, 128 of 1024 x 512 27-31 and 24-29; at 4 rows, in the same order, 4.3 and
// 8.7, 5-9 and 7, 66 and 79, 72 and 77, 68 and 70, 125-129 and 137, 25 and 24. The small ones gain most, and a few large ones lose.
constexpr int kExpertFewRows = 8;
hipError_t run_skinny_experts(DType in, int epi, const ExpertGemm& a, hipStream_t s);

// dz = dy f'(z) (gated: [dy u f'(g) | dy f(g)]) into dz [rows, P] (NULL: not stored; fn FN_NONE: dz is
// dy), and its column sums over pieces of at most dact_rows() rows of one expert, fp32, into
// sums [pieces][P] (NULL: not formed); P = 2N gated, else N. Pieces are 64 rows (8 rows a thread); where those
// would leave CUs idle, 16: a few rows after another are latency (1003 rows of 516 fp32: 8.2 -> 5.4 us).
constexpr int kDactRowsFew = 16, kDactRows = 64, kDactCols = 256;
inline int dact_rows(int64_t rows, int64_t N) {
  return rows / kDactRows * ((N + kDactCols - 1) / kDactCols) < 512 ? kDactRowsFew : kDactRows;
}
inline int64_t dact_pieces(int64_t rows, int64_t N, int64_t experts) {
  return rows / dact_rows(rows, N) + (rows < experts ? rows : experts) + 1;
}
hipError_t run_linear_dact(DType io, int gated, int fn, const void* dy, const void* preact, const int* offsets,
                           int experts, int64_t rows, int64_t N, void* dz, float* sums, hipStream_t s);
// The pieces' sums joined (BiasGrad, in `io`), as a launch of its own.
hipError_t run_linear_dbias(DType io, const BiasGrad& a, hipStream_t s);

// ---- router, sort, rows ---------------------------------------------------------------------------

hipError_t run_moe_route(DType dt, const void* logits, int64_t T, int E, int k, int sigmoid, int renorm, int* ids,
                         float* weights, hipStream_t s);
hipError_t run_moe_route_bwd(DType dt, const void* logits, const int* ids, const float* dweights, int64_t T, int E,
                             int k, int sigmoid, int renorm, void* dlogits, hipStream_t s);
// ws: moe_balance_parts x (E fp32 + E + 1 int32)
int moe_balance_parts(int64_t T, int E);
hipError_t run_moe_balance(DType dt, const void* logits, const int* ids, const uint8_t* mask, int64_t T, int E, int k,
                           int sigmoid, int* counts, float* shares, float* loss, void* ws, hipStream_t s);
hipError_t run_moe_balance_bwd(DType dt, const void* logits, const int* ids, const uint8_t* mask, const int* counts,
                               const float* dloss, const float* dweights, int64_t T, int E, int k, int sigmoid, int renorm,
                               void* dlogits, hipStream_t s);
size_t moe_sort_counts_bytes(int64_t n, int E);   // 0: one workgroup sorts them
hipError_t run_moe_sort(const int* ids, int64_t n, int E, int* offsets, int* row_of, int* slot_of, int* counts,
                        hipStream_t s);
// rows of `pieces` 16-byte pieces
hipError_t run_moe_gather(const void* x, const int* slot_of, const int* offsets, int n, int E, int k, int pieces,
                          void* xs, hipStream_t s);
hipError_t run_moe_combine(DType dt, const void* ys, const float* weights, const int* row_of, const int* offsets,
                           const void* residual, int T, int E, int k, int pieces, void* out, hipStream_t s);
hipError_t run_moe_combine_bwd(DType dt, const void* dout, const void* ys, const float* weights, const int* slot_of,
                               const int* offsets, int n, int E, int k, int pieces, void* dys, float* dweights,
                               hipStream_t s);

// ---- microscaled 4-bit floating point ------------------------------------------------------------------

hipError_t run_mx4_rows(DType dt, const void* x, int64_t batch, int64_t rows, int64_t cols, void* codes, void* scales,
                        hipStream_t s);
// row_codes: also what run_mx4_rows gives (16-bit types), x read once.
hipError_t run_mx4_columns(DType dt, const void* x, int64_t batch, int64_t rows, int64_t cols, void* codes, void* scales,
                           void* row_codes, void* row_scales, hipStream_t s);
hipError_t run_mx4_values(DType dt, const void* codes, const void* scales, int64_t batch, int64_t rows, int64_t K, void* out,
                          hipStream_t s);
// EPI_LIN or EPI_LIN_GATED, unsplit; tiles TILE_256x256, TILE_128x128 and TILE_64x64 (gated: 64 x 128)
hipError_t run_mx4_linear_bf16(int epi, TileShape tile, const Mx4Gemm& a, hipStream_t s);
hipError_t run_mx4_linear_f16(int epi, TileShape tile, const Mx4Gemm& a, hipStream_t s);
hipError_t run_mx4_linear_f32(int epi, TileShape tile, const Mx4Gemm& a, hipStream_t s);
// Few rows: 16 rows of one weight by 16 columns a workgroup. Taken up to kMxSkinnyRows rows of one weight, and up to
// kMxExpertRows an expert on average. Streamed and in tiles (us): 16 rows of 4096 x 11008 8.9 and 9.3, 32 14.8 and 9.3, 32 of
// 1024 x 1024 4.2 and 5.5, 16 of 2048 x 5504 gate and up 6.0 and 8.1; 64 experts of 2048 x 1376 gate and up, 2 rows each 42 and 48, 4 41
// and 45, 8 43 and 45, 16 48 and 45; 16 experts of 4096 x 1024, 16 rows each 11.3 and 9.5. The host does not know each expert's rows. Of
// the same gate and up, rows even, falling as 1 / rank, and all on four experts (whose weights are read anew for every 16 rows):
// 512 of 64 experts 46 and 47, 48 and 45, 23 and 9; 256 of 64 40 and 45, 36 and 35, 15 and 9; 1024 of 128 85 and 87, 94 and 87, 45 and 13.
constexpr int kMxSkinnyRows = 16, kMxExpertRows = 8;
hipError_t run_mx4_skinny(DType io, int gated, const Mx4Gemm& a, hipStream_t s);
// fp32 sums of a.splits parts of K, a.g.partial [splits][M][N]; B1: more rows of B from a.g.b_split on
hipError_t run_mx4_partial(TileShape tile, const Mx4Gemm& a, hipStream_t s);

// ---- norm ------------------------------------------------------------------------------------------

// Rows of `pieces` 16-byte pieces, d elements; wide: weight and bias are fp32, else of the rows' type.
hipError_t run_norm_fwd(DType dt, bool wide, const void* x, const void* res, const void* w, const void* b, int64_t rows,
                        int pieces, int64_t d, int layer, float eps, void* y, void* h, float* mean, float* rstd,
                        hipStream_t s);
// part: fp32 [norm_parts][2][d], where dw or db is asked for.
int norm_parts(int64_t rows, int pieces, bool fp32);
hipError_t run_norm_bwd(DType dt, bool wide, const void* dy, const void* h, const float* mean, const float* rstd,
                        const void* w, const void* dres, int64_t rows, int pieces, int64_t d, void* dx, void* dw,
                        void* db, int accumulate, float* part, hipStream_t s);

// out = alpha * sum_s partial[s] (fixed order), stored as `io` or added into fp32 (accumulate).
// Rows >= c_split go to C1 (row - c_split).
hipError_t run_splitk_reduce(DType io, const float* partial, int splits, int M, int N, void* C0,
                             void* C1, int64_t ldc, int c_split, float alpha, const float* dev0,
                             const float* dev1, int accumulate, hipStream_t s);

// Split-K finish of the gated up projection: g|u = alpha * sum of the fp32 partials [s][M][2H] in
// order; g|u -> preact [M, 2H] when non-NULL; a = act(g, u) -> a [M, H].
hipError_t run_gated_reduce(DType io, const float* partial, int splits, int M, int H, float alpha,
                            const float* dev0, const float* dev1, void* preact, void* a, float gate_mult,
                            int gate_inside, int fn, hipStream_t s);

// a[m][n] = act(g = pre[m][n], u = pre[m][H + n]) (gated), or post = f(alpha * pre); fn: ActFn.
hipError_t run_gated_act(DType io, const void* preact, void* a, int M, int H, float gate_mult,
                         int gate_inside, int fn, hipStream_t s);
hipError_t run_plain_act(DType io, const void* pre, void* post, int64_t n, float alpha,
                         const float* dev0, const float* dev1, int fn, hipStream_t s);

// Per-tensor e4m3 quantization: amax (into ws[0], from per-workgroup maxima in ws[64 ..
// 64 + kQuantizeParts)), then scale and codes. The workspace holds kQuantizeWsBytes.
constexpr int kQuantizeParts = 2048;
constexpr size_t kQuantizeWsBytes = 256 + kQuantizeParts * sizeof(float);
hipError_t run_quantize_e4m3(DType src_t, const void* src, int64_t n, void* dst, float* scale,
                             float* ws, hipStream_t s);
// Exact e4m3 -> bf16 widening (every e4m3 value is a bf16 value).
hipError_t run_dequant_e4m3_bf16(const void* src, void* dst, int64_t n, hipStream_t s);

// fp8 codes of a [rows, cols] row-major matrix (leading dimension ld_src elements), in row-major
// form (dst, leading dimension cols; may be NULL) and transposed (dst_t [cols, ld_t], ld_t >= rows
// a multiple of 16, columns rows .. ld_t-1 zero; may be NULL). src_t: DT_BF16 or DT_F32 (value
// v). relu_sq: quantize max(v, 0)^2 instead of v.
// e5m2: OCP E5M2 codes, else E4M3; code = fmt(v / *scale). cols must be a multiple of 16.
hipError_t run_quantize_fp8_2d(DType src_t, const void* src, int64_t rows, int64_t cols, int64_t ld_src,
                               int relu_sq, int e5m2, const float* scale, void* dst, void* dst_t,
                               int64_t ld_t, hipStream_t s);

// The fp8 weight-cache quantizer (row-major codes into dst, transposed into dst_t; either may be
// NULL): exact = 1 forms *scale from w's own amax (an amax pass first), exact = 0 from the per-tile
// amax the previous call recorded in tile_amax (weight_amax_slots(rows, cols) floats); both record
// w's per-tile amax there. src_t: DT_BF16 or DT_F32; cols a multiple of 16.
int64_t weight_amax_slots(int64_t rows, int64_t cols);
hipError_t run_quantize_weight_e4m3(DType src_t, const void* w, int64_t rows, int64_t cols, int exact, float* scale,
                                    float* tile_amax, void* dst, void* dst_t, int64_t ld_t, hipStream_t s);

}  // namespace gmlp
