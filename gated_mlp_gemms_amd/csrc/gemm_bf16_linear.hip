// bf16 linear layer y = res + act(x W^T + b) (launch table: gemm_dispatch16.hpp).
#include "gemm_dispatch16.hpp"

namespace gmlp {

hipError_t run_gemm_bf16_linear(int epi, TileShape tile, const GemmArgs& a, int grid, hipStream_t s) {
  return run_linear16<bf16>(epi, tile, a, grid, s);
}

}  // namespace gmlp
