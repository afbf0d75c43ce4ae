/*
 * Mixture-of-experts operators on AMD Instinct MI355X (gfx950), in the same library as mlp.h and
 * under its conventions: dense row-major device buffers owned by the caller, every check on the
 * host before any HIP call, work enqueued on `stream`, the statuses of mlp_status, the text of a
 * failed check from mlp_last_error(). Nothing is allocated and nothing synchronizes, so every
 * call can be captured into a HIP graph.
 *
 * One layer of E experts over T tokens, k experts a token (n = T k assignments, "slots": slot
 * t k + j is token t's j-th choice):
 *
 *   moe_route        scores [T, E] -> ids [T, k], weights [T, k]
 *   moe_balance      scores, ids -> tokens an expert, the loss that balances them
 *   moe_sort         ids -> offsets [E + 1], row_of [n], slot_of [n]   (slots in expert order)
 *   moe_gather       x [T, d] -> xs [n, d], row r = the token of slot slot_of[r]
 *   linear_fwd       experts > 0: rows of expert e times its weight, with bias and activation
 *   moe_combine      ys [n, d] -> out [T, d] = residual + sum_j weights[t][j] ys[row_of[t k + j]]
 *
 * and the gradients of each. linear_fwd / linear_bwd with experts = 0 are the same product with
 * one weight matrix: a linear layer with bias, activation and residual in its epilogue.
 *
 * Sizes may be zero where nothing is left to do (T, n, M = 0: pointers to empty tensors may then
 * be NULL). Rows are 16-byte aligned: d, K, N multiples of 8 (bf16, f16) or 4 (f32); every
 * buffer's address is 16-byte aligned (offsets, row_of, slot_of, ids: 4-byte).
 * int32 contents (ids, offsets, row_of, slot_of) are read on the device: an entry outside its
 * range never leads to an access out of bounds, as stated at each entry point.
 */
#ifndef GATED_MLP_MOE_H
#define GATED_MLP_MOE_H

#include "mlp.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Router scores: softmax over all E experts, or each expert's own sigmoid. */
typedef enum moe_score { MOE_SOFTMAX = 0, MOE_SIGMOID = 1 } moe_score;

#define MOE_MAX_EXPERTS 1024
#define MOE_MAX_CHOICES 16

/*
 * The k largest scores of each token, largest first, ties to the lowest expert (a NaN counts as
 * the largest), and their weights in fp32:
 *   softmax: p = softmax(logits[t]);  sigmoid: p = 1 / (1 + exp(-logits[t]));
 *   weights[t][j] = p[ids[t][j]], divided by the sum over the k chosen ones when renorm is 1.
 * logits [T, E] in dtype (f32, bf16, f16), scores of -inf allowed: such an expert is chosen last,
 * with weight 0; where every chosen probability is 0 all weights are 0 (never 0 / 0). A sigmoid counts as 0
 * below a score of -104 (2^-150); above, normalised weights are exact ratios also where the sigmoids
 * themselves are below fp32's range. A score of +inf has sigmoid 1; softmax over one is NaN.
 * 1 <= E <= MOE_MAX_EXPERTS, 1 <= k <= min(E, MOE_MAX_CHOICES).
 */
mlp_status moe_route(const void* logits, int dtype, int64_t T, int64_t E, int64_t k, int score, int renorm,
                     int32_t* ids, float* weights, void* stream);
/*
 * dlogits [T, E] (in dtype) = the gradient of moe_route's weights against dweights [T, k] (fp32),
 * the choice itself held fixed; p and the weights are formed again from logits. An id outside
 * [0, E) counts as not chosen.
 */
mlp_status moe_route_bwd(const void* logits, const int32_t* ids, const float* dweights, int dtype, int64_t T,
                         int64_t E, int64_t k, int score, int renorm, void* dlogits, void* stream);

/*
 * The load of each expert and the loss that balances it. Over the n tokens that count (mask [T], bytes: those
 * that are not 0; NULL: all), with the choices ids [T, k] held fixed,
 *   counts[e] = choices of expert e (an id outside [0, E) is none), counts[E] = n,
 *   shares[e] = mean of p[t][e],  p = softmax(logits[t]), or sigmoids divided by their sum over all E,
 *   loss[0] = E sum_e counts[e] / (n k) shares[e]        (1 when the load is even; 0 when n = 0).
 * counts [E + 1] int32; shares [E], loss [1] fp32, summed in fp32 in an order that depends on the sizes only. A token
 * whose scores are all -inf (sigmoid: below -104) has p = 0. What a token that does not count holds does not matter.
 * mask has any alignment.
 */
size_t moe_balance_workspace_bytes(int64_t T, int64_t E);   /* 0 for sizes moe_balance refuses, else >= 256 */
mlp_status moe_balance(const void* logits, const int32_t* ids, const uint8_t* mask, int dtype, int64_t T, int64_t E,
                       int64_t k, int score, int32_t* counts, float* shares, float* loss, void* workspace,
                       size_t workspace_bytes, void* stream);
/*
 * dlogits [T, E] (in dtype) = dloss[0] (fp32; NULL: 1) times the loss' gradient, through shares (counts do not depend
 * on the scores), 0 for a token that does not count; plus, with dweights [T, k] (fp32, NULL: none), what
 * moe_route_bwd gives for every token: the router's whole gradient in one pass, rounded once. counts is what
 * moe_balance wrote; ids is read with dweights only; renorm concerns dweights.
 */
mlp_status moe_balance_bwd(const void* logits, const int32_t* ids, const uint8_t* mask, const int32_t* counts,
                           const float* dloss, const float* dweights, int dtype, int64_t T, int64_t E, int64_t k,
                           int score, int renorm, void* dlogits, void* stream);

/*
 * Slots in expert order, a stable counting sort of the n ids: offsets[e] = number of slots of
 * experts below e (offsets[E] = all that are kept), slot_of[r] = the slot in row r, row_of its
 * inverse (row_of[slot_of[r]] = r). A slot whose id is outside [0, E) is dropped: it goes, in
 * slot order, behind the kept ones (rows offsets[E] .. n-1). n <= 2^30.
 */
size_t moe_sort_workspace_bytes(int64_t n, int64_t E);   /* 0 for sizes moe_sort refuses, else >= 256 */
mlp_status moe_sort(const int32_t* ids, int64_t n, int64_t E, int32_t* offsets, int32_t* row_of, int32_t* slot_of,
                    void* workspace, size_t workspace_bytes, void* stream);

/*
 * xs[r] = x[slot_of[r] / k] for the kept rows r < offsets[E], zeros behind them. x [T, d],
 * xs [T k, d], both dtype. A slot_of outside [0, T k) gives a row of zeros.
 */
mlp_status moe_gather(const void* x, const int32_t* slot_of, const int32_t* offsets, int dtype, int64_t T, int64_t E,
                      int64_t k, int64_t d, void* xs, void* stream);
/* dx[t] = sum over j of dxs[row_of[t k + j]], kept rows only, summed in fp32 in the order of j. */
mlp_status moe_gather_bwd(const void* dxs, const int32_t* row_of, const int32_t* offsets, int dtype, int64_t T,
                          int64_t E, int64_t k, int64_t d, void* dx, void* stream);
/*
 * out[t] = residual[t] + sum over j of weights[t][j] ys[row_of[t k + j]], kept rows only (a
 * dropped row is not read: what it holds does not matter), in fp32 in the order of j, rounded
 * once. residual may be NULL (zeros); out may be residual. weights [T, k] fp32.
 */
mlp_status moe_combine(const void* ys, const float* weights, const int32_t* row_of, const int32_t* offsets,
                       const void* residual, int dtype, int64_t T, int64_t E, int64_t k, int64_t d, void* out,
                       void* stream);
/*
 * Row by row, with s = slot_of[r] and t = s / k: for kept rows dys[r] = weights[s] dout[t] and
 * dweights[s] = dot(ys[r], dout[t]) (fp32 [T, k]); behind them zeros and 0. (The residual's
 * gradient is dout itself.)
 */
mlp_status moe_combine_bwd(const void* dout, const void* ys, const float* weights, const int32_t* slot_of,
                           const int32_t* offsets, int dtype, int64_t T, int64_t E, int64_t k, int64_t d, void* dys,
                           float* dweights, void* stream);

/* linear_desc.act: an mlp_act, or LINEAR_ACT_NONE (y = x W^T + b). */
#define LINEAR_ACT_NONE (-1)

typedef struct linear_desc {
  int64_t M;        /* rows of x (experts: all rows, dropped ones behind offsets[E] included), <= 2^29 */
  int64_t K;        /* width of x */
  int64_t N;        /* width of y */
  int32_t act;      /* mlp_act or LINEAR_ACT_NONE */
  int32_t dtype;    /* mlp_dtype of every tensor but offsets */
  int32_t experts;  /* 0: one weight [N, K]; E >= 1: weights [E, N, K], rows grouped by offsets */
} linear_desc;

typedef enum linear_phase { LINEAR_FWD = 0, LINEAR_BWD = 1 } linear_phase;

/* Bytes of workspace a phase needs (upper bound over every choice of optional arguments); 0 for
 * an invalid descriptor, else >= 256. Host only. */
size_t linear_workspace_bytes(const linear_desc* desc, int phase);

/*
 * z = x W^T + bias;  not gated: y = residual + f(z);
 * gated: g = x w^T + bias, u = x w_up^T + bias_up, y = residual + f(g) u.
 * Sums, bias, activation and residual in fp32, rounded once.
 *   x [M, K]; w (and w_up, iff gated) [N, K] or [E, N, K]; bias (bias_up iff gated) [N] or [E, N],
 *   NULL: none, both or neither; residual [M, N] or NULL (may be y);
 *   preact NULL or [M, N] = z, gated [M, 2N], row = [g | u], for linear_bwd;
 *   offsets [E + 1] iff experts: rows offsets[e] .. offsets[e+1]-1 are expert e's; rows behind
 *   offsets[E] get y = residual (zeros without one) and preact = 0. Offsets that are not
 *   monotone within [0, M] give wrong rows, never an access out of bounds.
 */
mlp_status linear_fwd(const linear_desc* desc, const void* x, const void* w, const void* w_up, const void* bias,
                      const void* bias_up, const void* residual, const int32_t* offsets, void* y, void* preact,
                      void* workspace, size_t workspace_bytes, void* stream);
/*
 * The backward against dy [M, N], from the preact that linear_fwd kept (NULL iff LINEAR_ACT_NONE):
 * dz = dy f'(z) (gated: dg = dy u f'(g), du = dy f(g)), rounded to dtype once, as the operand of
 *   dx [M, K] = dz W (dg w + du w_up),   dw / dw_up = dz^T x,   dbias / dbias_up = column sums of dz
 * (of dz before that rounding). Any of dx, dw (with dw_up), dbias (with dbias_up) may be NULL and
 * is then not formed. grad_accum 0: the weight and bias gradients are written in dtype; 1: they
 * are fp32 buffers that the new gradient is added to. Rows behind offsets[E] take no part and get
 * dx = 0; an expert without rows gets zeros (nothing is added with grad_accum).
 * (residual's gradient is dy itself.)
 */
mlp_status linear_bwd(const linear_desc* desc, const void* dy, const void* x, const void* w, const void* w_up,
                      const void* preact, const int32_t* offsets, void* dx, void* dw, void* dw_up, void* dbias,
                      void* dbias_up, int grad_accum, void* workspace, size_t workspace_bytes, void* stream);

/* Version of the declarations above. */
int moe_abi_version(void);

#ifdef __cplusplus
}
#endif
#endif /* GATED_MLP_MOE_H */
