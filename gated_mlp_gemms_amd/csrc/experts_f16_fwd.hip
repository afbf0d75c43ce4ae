// f16 products of the experts, forward (gemm_experts.hpp).
#include "gemm_experts.hpp"

namespace gmlp {

hipError_t run_expert_fwd_f16(int epi, TileShape tile, const ExpertGemm& a, hipStream_t s) {
  return expert_fwd16<f16>(epi, tile, a, s);
}

}  // namespace gmlp
