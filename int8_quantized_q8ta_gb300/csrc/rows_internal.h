// rows_internal.h -- host-side declarations of the operators for rows of one
// batch that go through different weights: the expert sort and its row moves
// (route_kernels.cu), and the grouped int8 contraction (tile_gemm.cu).
#pragma once

#include <cuda_runtime.h>

#include <cstdint>
#include <mutex>

#include "q8ta.h"
#include "q8ta_internal.h"

namespace q8 {

constexpr int kMaxExperts = 1024;  // the sort's per-warp counts fill shared memory

inline int64_t dtype_bytes(q8_dtype dt) { return dt == Q8_F32 ? 4 : dt == Q8_I8 ? 1 : 2; }

// A one-time set-up per device (kernel attributes).
class DeviceOnce {
 public:
  template <typename F>
  cudaError_t run(F&& f) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return f();
    std::lock_guard<std::mutex> lock(mu_);
    if (done_[dev]) return cudaSuccess;
    e = f();
    done_[dev] = e == cudaSuccess;
    return e;
  }

 private:
  std::mutex mu_;
  bool done_[64] = {false};
};

// launch_pdl with thread-block clusters of `cluster` CTAs along x.
template <typename... KArgs, typename... Args>
inline cudaError_t launch_pdl_cluster(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem,
                                      int cluster, cudaStream_t s, Args&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, static_cast<KArgs>(args)...);
  if (e != cudaSuccess) return e;
  return cudaGetLastError();
}

// ---- expert sort and row moves (route_kernels.cu) -------------------------
cudaError_t launch_expert_sort(const int32_t* ids, int64_t R, int E, int32_t* order,
                               int32_t* position, int32_t* offsets, cudaStream_t s);
cudaError_t launch_expert_gather(const void* x, int64_t T, int k, int64_t row_bytes,
                                 const int32_t* position, const int32_t* offsets, int E, void* xs,
                                 cudaStream_t s);
// y[t] = sum_j w[t,j] * z[position[t,j]]; w null: ones.
cudaError_t launch_expert_spread(const void* z, q8_dtype dt, const float* w, int64_t T, int k,
                                 int64_t H, const int32_t* position, void* y, cudaStream_t s);
cudaError_t launch_expert_combine_bwd(const void* dy, const void* z, q8_dtype dt, const float* w,
                                      int64_t T, int k, int64_t H, const int32_t* position,
                                      const int32_t* offsets, int E, void* dz, float* dw,
                                      cudaStream_t s);

}  // namespace q8
