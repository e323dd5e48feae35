// tile_gemm.cu -- the grouped contraction and the projection with adapters:
// the batch form of tile_gemm_kernel.cuh.
#include "tile_gemm_kernel.cuh"

namespace q8 {

cudaError_t launch_tile_gemm(TileParams p, const void* operand, q8_dtype out_dtype,
                             cudaStream_t s) {
  return launch_tiles<kFormBatch>(p, operand, out_dtype, s);
}

}  // namespace q8
