// token_kernels.cu -- rows with a scale for each token: float rows to int8 and
// back, the operands of the gradients, and the packing of gated weights.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cfloat>
#include <cstdint>
#include <type_traits>

#include "tile_device.cuh"
#include "token_device.cuh"
#include "token_internal.h"

namespace q8 {

namespace {

// ---------------------------------------------------------------------------
// a = max |x[m]|, s = a / 127, q = rint(x * (1 / s)): a row twice, once for its
// largest magnitude and once to round it.  A CTA has one row and keeps it in
// registers in between, so it comes from memory once; only rows beyond 4 items
// for each of 1,024 threads are read again (from L2).  Bytes bound it.
// ---------------------------------------------------------------------------
template <int DT, bool VEC, bool OP>
__global__ void __launch_bounds__(1024) quantize_token_kernel(const QuantizeJob job) {
  using Item = TokenItem<DT, VEC>;
  constexpr int U = VEC ? 4 : 16;
  __shared__ uint32_t tops[2][32];
  pdl_wait();
  pdl_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int warps = blockDim.x >> 5;
  if constexpr (OP)
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
         i < job.count_words; i += static_cast<int64_t>(gridDim.x) * blockDim.x)
      job.counts[i] = 0;
  const int64_t items = job.K / Item::kWidth;
  int turn = 0;
  for (int64_t m = blockIdx.x; m < job.M; m += gridDim.x, turn ^= 1) {
    const int64_t base = m * job.K;
    Item held[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t c = threadIdx.x + static_cast<int64_t>(u) * blockDim.x;
      if (c < items) held[u].load(job.x, base + c * Item::kWidth);
      else held[u].zero();
    }
    uint32_t top = 0;
#pragma unroll
    for (int u = 0; u < U; ++u) top = max(top, held[u].top());
    for (int64_t c = threadIdx.x + static_cast<int64_t>(U) * blockDim.x; c < items;
         c += blockDim.x) {
      Item it;
      it.load(job.x, base + c * Item::kWidth);
      top = max(top, it.top());
    }
    top = __reduce_max_sync(0xffffffffu, top);
    if (lane == 0) tops[turn][warp] = top;
    __syncthreads();
    top = __reduce_max_sync(0xffffffffu, lane < warps ? tops[turn][lane] : 0u);
    const TokenScale sc = token_scale(top);
    if (threadIdx.x == 0) job.scales[m] = sc.scale;
    const auto put = [&](const Item& it, int64_t c) {
      if constexpr (VEC) {
        const uint2 q = it.quantize(sc.inv);
        if (job.q != nullptr) *reinterpret_cast<uint2*>(job.q + base + c * 8) = q;
        if constexpr (OP)
          *reinterpret_cast<uint4*>(job.operand + ((c >> 3) * job.M + m) * 64 + (c & 7) * 8) =
              token_f16x8(q);
      } else {
        const int8_t q = it.quantize(sc.inv);
        if (job.q != nullptr) job.q[base + c] = q;
        if constexpr (OP)
          job.operand[((c >> 6) * job.M + m) * 64 + (c & 63)] =
              __half_as_ushort(__int2half_rn(q));
      }
    };
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t c = threadIdx.x + static_cast<int64_t>(u) * blockDim.x;
      if (c < items) put(held[u], c);
    }
    for (int64_t c = threadIdx.x + static_cast<int64_t>(U) * blockDim.x; c < items;
         c += blockDim.x) {
      Item it;
      it.load(job.x, base + c * Item::kWidth);
      put(it, c);
    }
    if constexpr (OP) {   // the last k-block's inputs past K
      const int64_t k = job.K + threadIdx.x;
      if (k < static_cast<int64_t>(job.KB) * 64)
        job.operand[((k >> 6) * job.M + m) * 64 + (k & 63)] = 0;
    }
  }
}

// Items 0 .. items - 1 of each of M rows, 32 * U at a time by a warp.
template <int U, typename F>
__device__ __forceinline__ void warp_segments(int64_t M, int64_t items, F&& f) {
  const int lane = threadIdx.x & 31;
  const int64_t segs = (items + U * 32 - 1) / (U * 32), units = M * segs;
  const int64_t t = (static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x) >> 5;
  const int64_t step = (static_cast<int64_t>(gridDim.x) * blockDim.x) >> 5;
  int64_t m = t / segs, seg = t - m * segs;
  const int64_t m_step = step / segs, seg_step = step - m_step * segs;
  for (int64_t u = t; u < units; u += step) {
    f(m, seg * U * 32 + lane);
    m += m_step;
    seg += seg_step;
    if (seg >= segs) {
      seg -= segs;
      ++m;
    }
  }
}

// out = float(q) * s, one rounding to the type.  VEC: 8 values an item.
template <int DT, bool VEC>
__global__ void __launch_bounds__(256) dequantize_token_kernel(const int8_t* q,
                                                               const float* scales, int64_t M,
                                                               int64_t K, void* out) {
  constexpr int U = 4, W = VEC ? 8 : 1;
  pdl_wait();
  pdl_launch_dependents();
  const int64_t items = K / W;
  warp_segments<U>(M, items, [&](int64_t m, int64_t c0) {
    const float s = scales[m];
    const int64_t base = m * K;
    uint2 w[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t c = c0 + u * 32;
      if (c < items) {
        if constexpr (VEC) w[u] = __ldcs(reinterpret_cast<const uint2*>(q + base + c * 8));
        else w[u].x = static_cast<uint8_t>(q[base + c]);
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t c = c0 + u * 32;
      if (c < items) {
        if constexpr (VEC) {
          float v[8];
#pragma unroll
          for (int j = 0; j < 8; ++j)
            v[j] = __fmul_rn(
                static_cast<float>(static_cast<int8_t>((j < 4 ? w[u].x : w[u].y) >> (8 * (j & 3)))),
                s);
          store_x8<DT>(out, base + c * 8, v);
        } else {
          store_one<DT>(out, base + c, __fmul_rn(static_cast<float>(static_cast<int8_t>(w[u].x)), s));
        }
      }
    }
  });
}

// ---------------------------------------------------------------------------
// Gradients.  A warp has 256 channels (their scales in registers) of several
// rows, so that the scales are read once for them.
// ---------------------------------------------------------------------------
constexpr int kGradRows = 16;

template <int DT, bool VEC, bool MASK>
__global__ void __launch_bounds__(256) grad_operand_kernel(const GradOperandJob job) {
  pdl_wait();
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
  const int64_t step = static_cast<int64_t>(gridDim.x) * blockDim.x;
  for (int64_t i = t; i < job.count_words; i += step) job.counts[i] = 0;
  const float rescale = job.rescale != nullptr ? *job.rescale : 1.0f;
  const int64_t chunks = static_cast<int64_t>(job.KB) * 8, segs = (chunks + 31) / 32;
  const int64_t groups = (job.M + kGradRows - 1) / kGradRows;
  const auto* dy = static_cast<const uint16_t*>(job.dy);
  const auto* y = static_cast<const uint16_t*>(job.y);
  for (int64_t u = t >> 5; u < groups * segs; u += step >> 5) {
    const int64_t seg = u % segs, m0 = u / segs * kGradRows;
    const int64_t c = seg * 32 + lane;
    if (c >= chunks) continue;
    float ws[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) ws[j] = c * 8 + j < job.N ? __ldg(job.ws + c * 8 + j) * rescale : 0.0f;
    const int64_t m1 = min(job.M, m0 + kGradRows);
    constexpr int U = 4;
    for (int64_t m = m0; m < m1; m += U) {
      uint4 v[U], w[U];
#pragma unroll
      for (int i = 0; i < U; ++i)
        if (m + i < m1) {
          v[i] = load_halves<VEC>(dy, (m + i) * job.N, c * 8, job.N);
          if constexpr (MASK) w[i] = load_halves<VEC>(y, (m + i) * job.N, c * 8, job.N);
        }
#pragma unroll
      for (int i = 0; i < U; ++i)
        if (m + i < m1) {
          const uint32_t d[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
          const uint32_t a[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
          uint32_t r[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            float lo = half_bits_to_float<DT>(d[j] & 0xffffu) * ws[2 * j];
            float hi = half_bits_to_float<DT>(d[j] >> 16) * ws[2 * j + 1];
            if constexpr (MASK) {
              if (!(half_bits_to_float<DT>(a[j] & 0xffffu) > 0.0f)) lo = 0.0f;
              if (!(half_bits_to_float<DT>(a[j] >> 16) > 0.0f)) hi = 0.0f;
            }
            r[j] = float_to_half_bits<DT>(lo) | (float_to_half_bits<DT>(hi) << 16);
          }
          *reinterpret_cast<uint4*>(job.dst + ((c >> 3) * job.M + m + i) * 64 + (c & 7) * 8) =
              make_uint4(r[0], r[1], r[2], r[3]);
        }
    }
  }
}

// One CTA: a few thousand scales.
__global__ void __launch_bounds__(1024) channel_norm_kernel(const float* __restrict__ ws, int64_t n,
                                                            float* __restrict__ norm) {
  __shared__ uint32_t tops[32];
  pdl_wait();
  pdl_launch_dependents();
  uint32_t top = 0;
#pragma unroll 4
  for (int64_t i = threadIdx.x; i < n; i += 1024)
    top = max(top, __float_as_uint(ws[i]) & 0x7fffffffu);
  top = __reduce_max_sync(0xffffffffu, top);
  if ((threadIdx.x & 31) == 0) tops[threadIdx.x >> 5] = top;
  __syncthreads();
  if (threadIdx.x < 32) {
    top = __reduce_max_sync(0xffffffffu, tops[threadIdx.x]);
    if (threadIdx.x == 0) {
      // zeros, infinities and NaN leave the scales as they are
      const int exponent = static_cast<int>(top >> 23);
      const int e = exponent == 0 || exponent == 255 ? 0 : min(max(exponent - 127, -100), 100);
      norm[0] = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
      norm[1] = __uint_as_float(static_cast<uint32_t>(127 + e) << 23);
    }
  }
}

// ---------------------------------------------------------------------------
// Gated weights, once, at load time: one 16-byte chunk per item, as in
// pack_tile_weight_kernel.
// ---------------------------------------------------------------------------
template <bool T>
__global__ void __launch_bounds__(256) pack_gated_kernel(const int8_t* __restrict__ gate,
                                                         const int8_t* __restrict__ up, int64_t N,
                                                         int64_t K, int64_t NB, int64_t KB,
                                                         uint4* __restrict__ dst) {
  pdl_wait();
  const int64_t total = NB * KB * 512;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; i < total;
       i += static_cast<int64_t>(gridDim.x) * blockDim.x) {
    const int64_t t = i >> 9, kb = t % KB;
    const int64_t row = t / KB * 128 + (i & 127), in0 = kb * 64 + ((i >> 7) & 3) * 16;
    uint32_t v[4] = {0x80808080u, 0x80808080u, 0x80808080u, 0x80808080u};
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      const int64_t pair = T ? in0 + j : row;          // the interleaved index
      const int64_t n = (pair >> 5) * 16 + (pair & 15), k = T ? row : in0 + j;
      if (n < N && k < K) {
        const uint32_t b = static_cast<uint8_t>(((pair & 16) ? up : gate)[n * K + k]);
        v[j / 4] ^= b << (8 * (j % 4));   // (over the zero's byte)
      }
    }
    dst[i] = make_uint4(v[0], v[1], v[2], v[3]);
  }
}
__global__ void larger_bound_kernel(int32_t* word) {
  pdl_wait();
  word[0] = max(word[0], word[1]);
}

bool on16(const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }

int blocks_for(int64_t warps) {
  return static_cast<int>(std::max<int64_t>(
      1, std::min<int64_t>((warps + 7) / 8, static_cast<int64_t>(device_sm_count()) * 8)));
}

// f(type, vectors) with the dtype and a truth value as constants
template <typename F>
cudaError_t by_type(q8_dtype dt, bool vec, F&& f) {
  const auto with = [&](auto t) { return vec ? f(t, std::true_type()) : f(t, std::false_type()); };
  switch (dt) {
    case Q8_F32: return with(std::integral_constant<int, Q8_F32>());
    case Q8_F16: return with(std::integral_constant<int, Q8_F16>());
    default: return with(std::integral_constant<int, Q8_BF16>());
  }
}

}  // namespace

cudaError_t launch_quantize_token(const QuantizeJob& job, q8_dtype dtype, cudaStream_t s) {
  const bool vec = job.K % 8 == 0 && on16(job.x) && reinterpret_cast<uintptr_t>(job.q) % 8 == 0;
  // One item a thread while there are few rows (its latency is what counts),
  // else four, whose loads are in flight together.
  const int64_t items = vec ? job.K / 8 : job.K;
  const int64_t each = job.M <= 2 * device_sm_count() ? 1 : vec ? 4 : 8;
  const int threads = static_cast<int>(
      std::min<int64_t>(1024, std::max<int64_t>(64, round_up((items + each - 1) / each, 32))));
  const int grid = static_cast<int>(std::min<int64_t>(job.M, INT32_MAX));
  return by_type(dtype, vec, [&](auto t, auto v) {
    constexpr int DT = decltype(t)::value;
    constexpr bool VEC = decltype(v)::value;
    return job.operand != nullptr
               ? launch_pdl(quantize_token_kernel<DT, VEC, true>, grid, threads, 0, s, job)
               : launch_pdl(quantize_token_kernel<DT, VEC, false>, grid, threads, 0, s, job);
  });
}

cudaError_t launch_dequantize_token(const int8_t* q, const float* scales, int64_t M, int64_t K,
                                    q8_dtype dtype, void* out, cudaStream_t s) {
  const bool vec = K % 8 == 0 && on16(out) && reinterpret_cast<uintptr_t>(q) % 8 == 0;
  const int64_t items = vec ? K / 8 : K;
  const int grid = blocks_for(M * ((items + 127) / 128));
  return by_type(dtype, vec, [&](auto t, auto v) {
    return launch_pdl(dequantize_token_kernel<decltype(t)::value, decltype(v)::value>, grid, 256, 0,
                      s, q, scales, M, K, out);
  });
}

cudaError_t launch_grad_operand(const GradOperandJob& job, q8_dtype dtype, cudaStream_t s) {
  const bool vec = job.N % 8 == 0 && on16(job.dy) && on16(job.y);
  const int64_t units = (job.M + kGradRows - 1) / kGradRows * ((job.KB * 8 + 31) / 32);
  const int grid = blocks_for(std::max<int64_t>(units, (job.count_words + 31) / 32));
  const auto go = [&](auto t, auto v) {
    constexpr int DT = decltype(t)::value;
    constexpr bool VEC = decltype(v)::value;
    return job.y != nullptr ? launch_pdl(grad_operand_kernel<DT, VEC, true>, grid, 256, 0, s, job)
                            : launch_pdl(grad_operand_kernel<DT, VEC, false>, grid, 256, 0, s, job);
  };
  const auto with = [&](auto t) { return vec ? go(t, std::true_type()) : go(t, std::false_type()); };
  return dtype == Q8_F16 ? with(std::integral_constant<int, Q8_F16>())
                         : with(std::integral_constant<int, Q8_BF16>());
}

cudaError_t launch_channel_norm(const float* ws, int64_t n, float* norm, cudaStream_t s) {
  return launch_pdl(channel_norm_kernel, 1, 1024, 0, s, ws, n, norm);
}

cudaError_t launch_pack_gated(const int8_t* gate, const int8_t* up, int64_t N, int64_t K,
                              bool transposed, uint8_t* dst, cudaStream_t s) {
  const int64_t pairs = gated_rows(N), rows = transposed ? K : pairs;
  // (the transposed weight's inputs reach to the end of the last block of 128
  // packed rows: that is how far the gated gradient's kernel writes)
  const int64_t NB = (rows + 127) / 128, KB = transposed ? (pairs + 127) / 128 * 2 : (K + 63) / 64;
  const int grid = blocks_for(NB * KB * 16);
  auto* to = reinterpret_cast<uint4*>(dst);
  return transposed ? launch_pdl(pack_gated_kernel<true>, grid, 256, 0, s, gate, up, N, K, NB, KB, to)
                    : launch_pdl(pack_gated_kernel<false>, grid, 256, 0, s, gate, up, N, K, NB, KB, to);
}

cudaError_t launch_larger_bound(int32_t* word, cudaStream_t s) {
  return launch_pdl(larger_bound_kernel, 1, 1, 0, s, word);
}

}  // namespace q8
