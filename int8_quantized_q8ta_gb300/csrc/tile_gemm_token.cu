// tile_gemm_token.cu -- products of rows with a scale for each token, and the
// gated pair of them: two forms of tile_gemm_kernel.cuh.
#include "tile_gemm_kernel.cuh"

namespace q8 {

cudaError_t launch_tile_token(TileParams p, const void* operand, q8_dtype out_dtype,
                              cudaStream_t s) {
  return launch_tiles<kFormToken>(p, operand, out_dtype, s);
}
cudaError_t launch_tile_gated(TileParams p, const void* operand, q8_dtype out_dtype,
                              cudaStream_t s) {
  return launch_tiles<kFormGated>(p, operand, out_dtype, s);
}

}  // namespace q8
