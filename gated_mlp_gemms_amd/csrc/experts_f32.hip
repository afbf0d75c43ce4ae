// fp32 products of the experts (gemm_experts.hpp).
#include "gemm_experts.hpp"

namespace gmlp {

hipError_t run_expert_fwd_f32(int epi, TileShape tile, const ExpertGemm& a, hipStream_t s) {
  if (tile == TILE_128x128_RING) return launch_expert_fwd<float, 128, 128, 4>(epi, a, s);
  if (tile != TILE_64x64_RING) return hipErrorInvalidValue;
  if (epi == EPI_LIN_GATED)
    hipLaunchKernelGGL((expert_fwd_kernel<float, 64, 128, EPI_LIN_GATED, 4>), dim3(a.grid), dim3(256), 0, s, a);
  else
    hipLaunchKernelGGL((expert_fwd_kernel<float, 64, 64, EPI_LIN, 4>), dim3(a.grid), dim3(256), 0, s, a);
  return hipGetLastError();
}
hipError_t run_expert_bwd_f32(TileShape tile, const ExpertBwd& a, hipStream_t s) {
  if (tile == TILE_128x128_RING) return launch_expert_bwd<float, 128, 128, 4>(a, s);
  if (tile == TILE_64x64_RING) return launch_expert_bwd<float, 64, 64, 4>(a, s);
  return hipErrorInvalidValue;
}

}  // namespace gmlp
