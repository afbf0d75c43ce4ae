// fp32 GEMMs of the linear layer on the DMA ring (gemm_dma.hpp), 128 x 128 and 64 x 64 tiles.
#include "gemm_dma.hpp"
#include "launch.hpp"

namespace gmlp {

template <int B>
static hipError_t ring(Layout layout, int epi, const GemmArgs& a, int grid, hipStream_t s) {
  switch (layout) {
    case NT:
      switch (epi) {
        case EPI_LIN: return launch_gemm_dma<float, float, B, B, true, true, EPI_LIN>(a, grid, s);
        case EPI_LIN_GATED:   // 64 rows only (linear_tiles)
          if constexpr (B == 64) return launch_gemm_dma<float, float, 64, 128, true, true, EPI_LIN_GATED>(a, grid, s);
          return hipErrorInvalidValue;
        case EPI_PARTIAL: return launch_gemm_dma<float, float, B, B, true, true, EPI_PARTIAL>(a, grid, s);
        default: return hipErrorInvalidValue;
      }
    case NN:
      switch (epi) {
        case EPI_STORE: return launch_gemm_dma<float, float, B, B, true, false, EPI_STORE>(a, grid, s);
        case EPI_PARTIAL: return launch_gemm_dma<float, float, B, B, true, false, EPI_PARTIAL>(a, grid, s);
        default: return hipErrorInvalidValue;
      }
    case TN:
      switch (epi) {
        case EPI_STORE: return launch_gemm_dma<float, float, B, B, false, false, EPI_STORE>(a, grid, s);
        case EPI_PARTIAL: return launch_gemm_dma<float, float, B, B, false, false, EPI_PARTIAL>(a, grid, s);
        default: return hipErrorInvalidValue;
      }
  }
  return hipErrorInvalidValue;
}

hipError_t run_gemm_f32_ring(Layout layout, int epi, TileShape tile, const GemmArgs& a, int grid, hipStream_t s) {
  if (tile == TILE_128x128_RING) return ring<128>(layout, epi, a, grid, s);
  if (tile == TILE_64x64) return ring<64>(layout, epi, a, grid, s);
  return hipErrorInvalidValue;
}

}  // namespace gmlp
