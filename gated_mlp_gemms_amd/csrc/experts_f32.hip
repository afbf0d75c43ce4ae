// fp32 products of the experts (gemm_experts.hpp).
#include "gemm_experts.hpp"

namespace gmlp {

hipError_t run_expert_fwd_f32(int epi, TileShape tile, const ExpertGemm& a, hipStream_t s) {
  if (tile == TILE_128x128_RING && epi == EPI_LIN) {   // (gated: 64 rows only, linear_tiles)
    hipLaunchKernelGGL((expert_fwd_kernel<float, 128, 128, EPI_LIN, 4>), dim3(a.grid), dim3(256), 0, s, a);
    return hipGetLastError();
  }
  if (tile == TILE_64x64) return launch_expert_fwd_small<float>(epi, a, s);
  return hipErrorInvalidValue;
}
hipError_t run_expert_bwd_f32(TileShape tile, const ExpertBwd& a, hipStream_t s) {
  if (tile == TILE_128x128_RING) return launch_expert_bwd<float, 128, 128, 4>(a, s);
  if (tile == TILE_64x64) return launch_expert_bwd<float, 64, 64, 4>(a, s);
  return hipErrorInvalidValue;
}

}  // namespace gmlp
