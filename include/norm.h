/*
 * The norm in front of a layer on AMD Instinct MI355X (gfx950), in the same library as mlp.h and
 * under its conventions: dense row-major device buffers owned by the caller, every check on the
 * host before any HIP call, work enqueued on `stream`, the statuses of mlp_status, the text of a
 * failed check from mlp_last_error(). Nothing is allocated and nothing synchronizes, so every
 * call can be captured into a HIP graph.
 *
 * Rows are 16-byte aligned: d a multiple of 8 (bf16, f16) or 4 (f32); every buffer's address is
 * 16-byte aligned (mean, rstd: 4-byte). M may be 0 (pointers to empty tensors may then be NULL).
 */
#ifndef GATED_MLP_NORM_H
#define GATED_MLP_NORM_H

#include "mlp.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Layer norm, or RMS norm: the same without the mean (m = 0). */
typedef enum norm_kind { NORM_LAYER = 0, NORM_RMS = 1 } norm_kind;

typedef struct norm_desc {
  int64_t M;        /* rows, <= 2^30 */
  int64_t d;        /* width, < 2^25 */
  int32_t dtype;    /* mlp_dtype of the rows */
  int32_t wdtype;   /* of weight and bias: dtype, or MLP_F32 */
  int32_t kind;     /* norm_kind */
  float eps;        /* >= 0, finite */
} norm_desc;

/*
 * h = x + residual (residual NULL: h = x), rounded to dtype; over a row's d elements
 *   m = mean(h) (RMS: 0),  s = 1 / sqrt(mean((h - m)^2) + eps),  y = (h - m) s weight + bias,
 * statistics and sums in fp32 from the rounded h, the squares of the differences summed after the mean is known; y rounded
 * once.
 *   x, residual, y [M, d]; weight, bias [d], NULL: 1 and 0 (a bias without a weight is refused);
 *   h_out NULL or [M, d], with a residual only: receives h (it may be x or residual);
 *   mean (layer norm only), rstd NULL or [M] fp32: receive m and s, for norm_bwd.
 */
mlp_status norm_fwd(const norm_desc* desc, const void* x, const void* residual, const void* weight, const void* bias,
                    void* y, void* h_out, float* mean, float* rstd, void* stream);

/* Bytes of workspace norm_bwd needs; 0 for sizes it refuses, else >= 256. Host only. */
size_t norm_workspace_bytes(int64_t M, int64_t d);

/*
 * The backward against dy [M, d], with h what the norm was taken of and mean, rstd what norm_fwd
 * gave: with g = dy weight, n = (h - m) s,
 *   dx = s (g - mean(g) - n mean(g n)) + dresidual    (RMS: without mean(g)),
 *   dweight = sum over the rows of dy n,   dbias = sum over the rows of dy,
 * in fp32, each rounded once. dx is the gradient of h, so of x and of residual alike; dresidual
 * (NULL: 0) is what else reached h, and dx may be dresidual. mean is NULL iff RMS. Any of dx, dweight,
 * dbias may be NULL and is then not formed. grad_accum 0: dweight and dbias are written in
 * wdtype; 1: they are fp32 buffers that the new gradient is added to. The sums' order depends on
 * the sizes only. M = 0: the gradients are 0 (nothing is added with grad_accum).
 */
mlp_status norm_bwd(const norm_desc* desc, const void* dy, const void* h, const float* mean, const float* rstd,
                    const void* weight, const void* dresidual, void* dx, void* dweight, void* dbias, int grad_accum,
                    void* workspace, size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif
#endif /* GATED_MLP_NORM_H */
