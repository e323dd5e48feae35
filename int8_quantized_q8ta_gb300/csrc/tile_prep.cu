// tile_prep.cu -- what the grouped int8 contraction (tile_gemm.cu) reads:
// load-time packing of weights, and the token operand.  Bandwidth-bound.
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "rows_internal.h"
#include "tile_device.cuh"

namespace q8 {

namespace {

int blocks_for(int64_t items) {
  return static_cast<int>(std::max<int64_t>(
      1, std::min<int64_t>((items + 255) / 256, static_cast<int64_t>(device_sm_count()) * 8)));
}

// One 16-byte chunk (a row's 16 inputs) per item.
__global__ void __launch_bounds__(256) pack_tile_weight_kernel(const int8_t* __restrict__ w,
                                                               int64_t E, int64_t N, int64_t K,
                                                               int64_t NB, int64_t KB,
                                                               uint4* __restrict__ dst) {
  pdl_wait();
  const int64_t total = E * NB * KB * 512;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; i < total;
       i += static_cast<int64_t>(gridDim.x) * blockDim.x) {
    const int64_t row = i & 127, c = (i >> 7) & 3;
    int64_t t = i >> 9;
    const int64_t kb = t % KB;
    t /= KB;
    const int64_t n = (t % NB) * 128 + row, e = t / NB, k0 = kb * 64 + c * 16;
    uint32_t v[4] = {0x80808080u, 0x80808080u, 0x80808080u, 0x80808080u};
    if (n < N) {
      const int8_t* src = w + (e * N + n) * K;
#pragma unroll
      for (int j = 0; j < 16; ++j)
        if (k0 + j < K) {
          const uint32_t b = static_cast<uint8_t>(src[k0 + j]);   // 0x80 ^ b replaces the zero's byte
          v[j / 4] ^= b << (8 * (j % 4));
        }
    }
    dst[i] = make_uint4(v[0], v[1], v[2], v[3]);
  }
}

// Eight inputs of one row per item.
__device__ __forceinline__ void operand_item(const OperandJob& job, int64_t i, bool vec,
                                             __half2 minus) {
  // consecutive items: the 8 chunks of a row's 64 inputs, then the next k-block
  const int per_row = job.KB * 8;
  const int64_t s = i / per_row;
  const int c = static_cast<int>(i - s * per_row);
  int64_t row = s;
  if (job.order != nullptr) {
    const int slot = __ldg(job.order + s);
    if (slot < 0) return;
    row = slot / job.k;
  }
  if (row >= job.x_rows) return;
  const int8_t* src = job.x + row * job.K + c * 8;
  uint2 w = make_uint2(0, 0);
  if (vec && c * 8 < job.K) {
    w = __ldg(reinterpret_cast<const uint2*>(src));
  } else {
    uint32_t v[2] = {0, 0};
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (c * 8 + j < job.K)
        v[j / 4] |= static_cast<uint32_t>(static_cast<uint8_t>(__ldg(src + j))) << (8 * (j % 4));
    w = make_uint2(v[0], v[1]);
  }
  // inputs past K give -zp here; their weights are zero
  w.x ^= 0x80808080u;
  w.y ^= 0x80808080u;
  uint4 o;
  o.x = biased_to_f16x2(w.x, 0x4140, minus);
  o.y = biased_to_f16x2(w.x, 0x4342, minus);
  o.z = biased_to_f16x2(w.y, 0x4140, minus);
  o.w = biased_to_f16x2(w.y, 0x4342, minus);
  job.dst[(static_cast<int64_t>(c >> 3) * job.R + s) * 8 + (c & 7)] = o;
}

__global__ void __launch_bounds__(256) tile_operand_kernel(const OperandJob job, bool vec) {
  pdl_wait();
  pdl_launch_dependents();
  const int64_t t = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
  const int64_t step = static_cast<int64_t>(gridDim.x) * blockDim.x;
  for (int64_t i = t; i < job.count_words; i += step) job.counts[i] = 0;
  // x - zp = (1024 + u) - (1152 + zp): integers below 2048, exact in f16
  const __half2 minus = __half2half2(__int2half_rn(1152 + job.zp));
  const int64_t total = static_cast<int64_t>(job.R) * job.KB * 8;
  for (int64_t i = t; i < total; i += step) operand_item(job, i, vec, minus);
}

bool rows_vec8(const OperandJob& job) {
  return job.K % 8 == 0 && reinterpret_cast<uintptr_t>(job.x) % 8 == 0;
}

}  // namespace

cudaError_t launch_pack_tile_weight(const int8_t* w, int64_t E, int64_t N, int64_t K, uint8_t* dst,
                                    cudaStream_t s) {
  const int64_t NB = (N + 127) / 128, KB = (K + 63) / 64;
  return launch_pdl(pack_tile_weight_kernel, blocks_for(E * NB * KB * 512), 256, 0, s, w, E, N, K,
                    NB, KB, reinterpret_cast<uint4*>(dst));
}

cudaError_t launch_tile_operand(const OperandJob& job, cudaStream_t s) {
  return launch_pdl(tile_operand_kernel,
                    blocks_for(std::max<int64_t>(static_cast<int64_t>(job.R) * job.KB * 8,
                                                 job.count_words)),
                    256, 0, s, job, rows_vec8(job));
}

}  // namespace q8
