// 16-bit GEMMs of the linear layer in 64 x 64 tiles (64 x 128 gated): small products, whose larger tiles
// would leave most CUs idle.
#include "gemm_dispatch16.hpp"

namespace gmlp {

template <typename T>
static hipError_t small(DType io, Layout layout, int epi, const GemmArgs& a, int grid, hipStream_t s) {
  switch (layout) {
    case NT:
      if (epi == EPI_LIN) return launch_gemm_dma<T, T, 64, 64, true, true, EPI_LIN>(a, grid, s);
      if (epi == EPI_LIN_GATED) return launch_gemm_dma<T, T, 64, 128, true, true, EPI_LIN_GATED>(a, grid, s);
      if (epi == EPI_PARTIAL) return launch_gemm_dma<T, float, 64, 64, true, true, EPI_PARTIAL>(a, grid, s);
      return hipErrorInvalidValue;
    case NN:
      if (epi == EPI_STORE) return launch_gemm_dma<T, T, 64, 64, true, false, EPI_STORE>(a, grid, s);
      if (epi == EPI_PARTIAL) return launch_gemm_dma<T, float, 64, 64, true, false, EPI_PARTIAL>(a, grid, s);
      return hipErrorInvalidValue;
    case TN:
      if (epi == EPI_STORE && io == DT_F32) return launch_gemm_dma<T, float, 64, 64, false, false, EPI_STORE>(a, grid, s);
      if (epi == EPI_STORE) return launch_gemm_dma<T, T, 64, 64, false, false, EPI_STORE>(a, grid, s);
      if (epi == EPI_PARTIAL) return launch_gemm_dma<T, float, 64, 64, false, false, EPI_PARTIAL>(a, grid, s);
      return hipErrorInvalidValue;
  }
  return hipErrorInvalidValue;
}

hipError_t run_gemm_small16(DType in, DType io, Layout layout, int epi, const GemmArgs& a, int grid, hipStream_t s) {
  if (in == DT_BF16) return small<bf16>(io, layout, epi, a, grid, s);
  if (in == DT_F16) return small<f16>(io, layout, epi, a, grid, s);
  return hipErrorInvalidValue;
}

}  // namespace gmlp
