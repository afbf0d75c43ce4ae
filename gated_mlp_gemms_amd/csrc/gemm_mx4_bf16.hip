// Products of microscaled 4-bit operands with outputs in bf16.
#include "gemm_mx4.hpp"

namespace gmlp {

hipError_t run_mx4_linear_bf16(int epi, TileShape tile, const Mx4Gemm& a, hipStream_t s) { return mx_linear<bf16>(epi, tile, a, s); }

}  // namespace gmlp
