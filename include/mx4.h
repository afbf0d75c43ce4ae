/*
 * Microscaled 4-bit floating point (OCP MXFP4) on AMD Instinct MI355X (gfx950), in the same library
 * as mlp.h and under its conventions: dense row-major device buffers owned by the caller, every
 * check on the host before any HIP call, work enqueued on `stream`, the statuses of mlp_status, the
 * text of a failed check from mlp_last_error(). Nothing is allocated and nothing synchronizes, so
 * every call can be captured into a HIP graph.
 *
 * 32 values that follow one another share a scale 2^(s - 127), s a byte (255: NaN, the whole block is
 * NaN); a value is its scale times an e2m1 code, +-{0, 0.5, 1, 1.5, 2, 3, 4, 6}, bit 3 the sign.
 *
 * A matrix of `rows` rows of K values (K a multiple of 32, blocks along the row) is held as
 *   codes   [rows][K / 2] bytes, value 2 i in the low half of byte i;
 *   scales  [mx4_planes(K)][mx4_scale_rows(rows)][8] bytes: block b of row r is at [b / 8][r][b % 8],
 *           blocks behind the last are 0, rows behind the last are not read as data.
 * A product's tile reads 256 values of its rows at a time, whose scales are one run of memory that way.
 * A batch of matrices is one after another. Buffers' addresses are 16-byte aligned.
 *
 * Size limits (MLP_ERR_UNSUPPORTED, before any HIP call): rows and M <= 2^29, columns, K and N (gated: 2 N) < 2^25,
 * a batch <= 65535, MOE_MAX_EXPERTS experts, 2^37 elements a matrix (all experts' weights are one); and a product
 * must fit a launch: its tiles, of 256 x 256 at most (gated: 256 x 128), are fewer than 2^24 (only many experts with
 * millions of columns have more).
 */
#ifndef GATED_MLP_MX4_H
#define GATED_MLP_MX4_H

#include "moe.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ceil(K / 256), and rows rounded up to the next larger multiple of 4. Host only. */
int64_t mx4_planes(int64_t K);
int64_t mx4_scale_rows(int64_t rows);

/*
 * x [batch][rows][cols] (dtype: f32, bf16, f16) to blocks along the rows (codes and scales; cols a multiple of
 * 32) and / or to blocks of the transposed matrix [batch][cols][deep], deep = rows rounded up to a
 * multiple of 32, zeros behind the last row (codes_t and scales_t; cols a multiple of 8, f32: 4): the
 * operands of a product along cols and of one along rows. codes and scales are both given or both NULL, as are
 * codes_t and scales_t. A block's scale is 2^(floor(log2 max|x|) - 2), at least 2^-127 (also of a block of
 * zeros); its values are rounded to the nearest code, ties to the even one, and saturate at 6; a NaN or an infinity in a
 * block makes its scale NaN.
 */
mlp_status mx4_quantize(const void* x, int dtype, int64_t batch, int64_t rows, int64_t cols, void* codes, void* scales,
                        void* codes_t, void* scales_t, void* stream);

/* out [batch][rows][K] (dtype) = the values that codes and scales stand for, rounded to dtype. */
mlp_status mx4_dequantize(const void* codes, const void* scales, int dtype, int64_t batch, int64_t rows, int64_t K,
                          void* out, void* stream);

/*
 * linear_fwd (moe.h) on 4-bit operands: the same formula, on the values that x [M, K] and w (w_up iff gated)
 * [N, K] or [E, N, K] stand for; desc->dtype is that of bias, residual, y and preact. Products and sums in fp32,
 * rounded once. K a multiple of 32, N of 8. With blocks of the transposed matrices it gives the products of the backward of a layer
 * without an activation, too: dx [M, K] = dy (W^T)^T from dy's blocks along N and W^T's (of experts [E, K, N]), and of one weight
 * dW [N, K] = dy^T (x^T)^T from the transposed blocks of both (rows that were added as zeros add nothing; an expert's
 * rows do not end where blocks do). Neither dy through an activation nor a bias' gradient is formed. residual may be y, which
 * adds to it.
 */
size_t mx4_linear_workspace_bytes(const linear_desc* desc);   /* 0 for what mx4_linear_fwd refuses, else >= 256 */
mlp_status mx4_linear_fwd(const linear_desc* desc, const void* x, const void* x_scales, const void* w,
                          const void* w_scales, const void* w_up, const void* w_up_scales, const void* bias,
                          const void* bias_up, const void* residual, const int32_t* offsets, void* y, void* preact,
                          void* workspace, size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif
#endif /* GATED_MLP_MX4_H */
