// fp32 products of the experts, and the fp32 linear layer (gemm_experts.hpp, gemm_kernel.hpp).
#include "gemm_experts.hpp"

namespace gmlp {

hipError_t run_expert_fwd_f32(int epi, const ExpertGemm& a, hipStream_t s) {
  return launch_expert_fwd<float, 128, 128, 4>(epi, a, s);
}
hipError_t run_expert_bwd_f32(const ExpertBwd& a, hipStream_t s) { return launch_expert_bwd<float, 128, 128, 4>(a, s); }

hipError_t run_gemm_f32_linear(int epi, const GemmArgs& a, int grid, hipStream_t s) {
  if (epi == EPI_LIN_GATED) return launch_gemm<float, float, 128, 128, true, true, EPI_LIN_GATED>(a, grid, s);
  if (epi == EPI_LIN) return launch_gemm<float, float, 128, 128, true, true, EPI_LIN>(a, grid, s);
  return hipErrorInvalidValue;
}

}  // namespace gmlp
