// Products of microscaled 4-bit operands with outputs in f32, and the partial sums of every type.
#include "gemm_mx4.hpp"

namespace gmlp {

hipError_t run_mx4_linear_f32(int epi, TileShape tile, const Mx4Gemm& a, hipStream_t s) { return mx_linear<float>(epi, tile, a, s); }

hipError_t run_mx4_partial(TileShape tile, const Mx4Gemm& a, hipStream_t s) {
  switch (tile) {
    case TILE_256x256: return launch_mx<float, 256, 256, EPI_PARTIAL>(a, s);
    case TILE_128x128: return launch_mx<float, 128, 128, EPI_PARTIAL>(a, s);
    case TILE_64x64: return launch_mx<float, 64, 64, EPI_PARTIAL>(a, s);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace gmlp
