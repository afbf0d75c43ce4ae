// C-ABI of the norm (norm.h): argument checks, all on the host before any HIP call, and the launches.
#include <algorithm>
#include <math.h>

#include "host_api.hpp"
#include "norm.h"

using namespace gmlp;

namespace {

mlp_status check_size(int64_t M, int64_t d) {
  if (M < 0) return fail(MLP_ERR_INVALID_ARG, "M = %lld rows", (long long)M);
  if (d < 1) return fail(MLP_ERR_INVALID_ARG, "d = %lld must be >= 1", (long long)d);
  if (M > (int64_t)1 << 30) return fail(MLP_ERR_UNSUPPORTED, "M is above 2^30");
  if (d >= (int64_t)1 << 25) return fail(MLP_ERR_UNSUPPORTED, "d is 2^25 or more");
  if (M > ((int64_t)1 << 37) / d) return fail(MLP_ERR_UNSUPPORTED, "M d is above 2^37 elements");
  return MLP_OK;
}

mlp_status check_norm(const norm_desc* q) {
  if (!q) return fail(MLP_ERR_INVALID_ARG, "desc is NULL");
  if (q->dtype != MLP_F32 && q->dtype != MLP_BF16 && q->dtype != MLP_F16)
    return fail(MLP_ERR_INVALID_ARG, "dtype %d is not an mlp_dtype", q->dtype);
  if (q->wdtype != q->dtype && q->wdtype != MLP_F32)
    return fail(MLP_ERR_INVALID_ARG, "wdtype %d is neither dtype (%d) nor MLP_F32", q->wdtype, q->dtype);
  if (q->kind != NORM_LAYER && q->kind != NORM_RMS) return fail(MLP_ERR_INVALID_ARG, "kind %d is not a norm_kind", q->kind);
  if (!(q->eps >= 0.0f) || !isfinite(q->eps)) return fail(MLP_ERR_INVALID_ARG, "eps must be finite and >= 0");
  MLP_TRY(check_size(q->M, q->d));
  const int v = q->dtype == MLP_F32 ? 4 : 8;
  if (q->d % v) return fail(MLP_ERR_ALIGNMENT, "d must be a multiple of %d (16-byte rows)", v);
  return MLP_OK;
}

mlp_status need_rows(const void* p, int64_t rows, const char* name, bool align16 = true) {
  return rows == 0 && !p ? MLP_OK : need_ptr(p, name, align16);
}
mlp_status optional(const void* p, const char* name, bool align16 = true) { return p ? need_ptr(p, name, align16) : MLP_OK; }

int pieces_of(const norm_desc* q) { return (int)(q->d * esize(q->dtype) / 16); }
hipStream_t stream_of(void* s) { return reinterpret_cast<hipStream_t>(s); }

}  // namespace

extern "C" {

mlp_status norm_fwd(const norm_desc* q, const void* x, const void* residual, const void* weight, const void* bias,
                    void* y, void* h_out, float* mean, float* rstd, void* stream) {
  MLP_TRY(check_norm(q));
  MLP_TRY(need_rows(x, q->M, "x"));
  MLP_TRY(need_rows(y, q->M, "y"));
  MLP_TRY(optional(residual, "residual"));
  MLP_TRY(optional(weight, "weight"));
  MLP_TRY(optional(bias, "bias"));
  if (bias && !weight) return fail(MLP_ERR_INVALID_ARG, "a bias needs a weight");
  MLP_TRY(optional(h_out, "h_out"));
  if (h_out && !residual && q->M > 0) return fail(MLP_ERR_INVALID_ARG, "h_out needs a residual (without one h is x)");
  if (mean && q->kind == NORM_RMS) MLP_TRY(need_null(mean, "mean", "for RMS norm"));
  MLP_TRY(optional(mean, "mean", false));
  MLP_TRY(optional(rstd, "rstd", false));
  if (q->M == 0) return MLP_OK;
  return hip_status(run_norm_fwd(dtype_of(q->dtype), q->wdtype == MLP_F32, x, residual, weight, bias, q->M, pieces_of(q),
                                 q->d, q->kind == NORM_LAYER, q->eps, y, h_out, mean, rstd, stream_of(stream)),
                    "norm_fwd");
}

size_t norm_workspace_bytes(int64_t M, int64_t d) {
  if (check_size(M, d) != MLP_OK) return 0;
  // the parts of either element size (a row has d / 4 pieces at most, d / 8 at least)
  const int parts = std::max(norm_parts(M, (int)((d + 3) / 4), true), norm_parts(M, (int)((d + 7) / 8), false));
  return std::max<size_t>(round_up((size_t)parts * 2 * (size_t)d * sizeof(float)), kAlign);
}

mlp_status norm_bwd(const norm_desc* q, const void* dy, const void* h, const float* mean, const float* rstd,
                    const void* weight, const void* dresidual, void* dx, void* dweight, void* dbias, int grad_accum,
                    void* workspace, size_t workspace_bytes, void* stream) {
  MLP_TRY(check_norm(q));
  if (grad_accum != 0 && grad_accum != 1) return fail(MLP_ERR_INVALID_ARG, "grad_accum must be 0 or 1");
  MLP_TRY(need_rows(dy, q->M, "dy"));
  MLP_TRY(need_rows(h, q->M, "h"));
  if (q->kind == NORM_RMS) MLP_TRY(need_null(mean, "mean", "for RMS norm"));
  else MLP_TRY(need_rows(mean, q->M, "mean", false));
  MLP_TRY(need_rows(rstd, q->M, "rstd", false));
  MLP_TRY(optional(weight, "weight"));
  MLP_TRY(optional(dresidual, "dresidual"));
  MLP_TRY(optional(dx, "dx"));
  if (dresidual && !dx) return fail(MLP_ERR_INVALID_ARG, "dresidual needs a dx to be added to");
  MLP_TRY(optional(dweight, "dweight"));
  MLP_TRY(optional(dbias, "dbias"));
  const bool sums = dweight || dbias;
  if (sums) {
    MLP_TRY(need_ptr(workspace, "workspace"));
    const size_t need = norm_workspace_bytes(q->M, q->d);
    if (workspace_bytes < need)
      return fail(MLP_ERR_WORKSPACE, "workspace of %zu bytes is smaller than the %zu needed", workspace_bytes, need);
  }
  if (!sums && (q->M == 0 || !dx)) return MLP_OK;
  return hip_status(run_norm_bwd(dtype_of(q->dtype), q->wdtype == MLP_F32, dy, h, mean, rstd, weight, dresidual, q->M,
                                 pieces_of(q), q->d, dx, dweight, dbias, grad_accum, static_cast<float*>(workspace),
                                 stream_of(stream)),
                    "norm_bwd");
}

}  // extern "C"
