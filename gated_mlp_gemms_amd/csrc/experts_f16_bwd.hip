// f16 products of the experts, backward (gemm_experts.hpp).
#include "gemm_experts.hpp"

namespace gmlp {

hipError_t run_expert_bwd_f16(TileShape tile, const ExpertBwd& a, hipStream_t s) {
  return expert_bwd16<f16>(tile, a, s);
}

}  // namespace gmlp
