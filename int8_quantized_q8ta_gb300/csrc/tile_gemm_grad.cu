// tile_gemm_grad.cu -- the gradients through int8 weights: the gated pair
// computed again up to its two gradients, and 16-bit float rows times the
// transposed weight.  Two forms of tile_gemm_kernel.cuh.
#include "tile_gemm_kernel.cuh"

namespace q8 {

cudaError_t launch_tile_gated_grad(TileParams p, const void* operand, q8_dtype dtype,
                                   cudaStream_t s) {
  return launch_tiles<kFormGatedGrad>(p, operand, dtype, s);
}
cudaError_t launch_tile_grad(TileParams p, const void* operand, q8_dtype dtype, cudaStream_t s) {
  return launch_tiles<kFormGrad>(p, operand, dtype, s);
}

}  // namespace q8
