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
// Gradients: rows of f16 for the product with the transposed weight, each under
// a power of two of its own (see row_power).
// ---------------------------------------------------------------------------
__device__ __forceinline__ uint32_t magnitude(float v) { return __float_as_uint(v) & 0x7fffffffu; }

// The largest of a CTA's threads' words, by every thread; `slots` is not used
// again before the next barrier but one.
__device__ __forceinline__ uint32_t block_max(uint32_t v, uint32_t (&slots)[32]) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  v = __reduce_max_sync(0xffffffffu, v);
  if (lane == 0) slots[warp] = v;
  __syncthreads();
  return __reduce_max_sync(0xffffffffu, lane < static_cast<int>(blockDim.x >> 5) ? slots[lane] : 0u);
}

// The largest magnitude of a CTA's share of n floats, four on a 16-byte
// boundary at a time where they lie so.
__device__ __forceinline__ uint32_t top_of(const float* v, int64_t n) {
  uint32_t top = 0;
  const int64_t head = min(n, static_cast<int64_t>((16 - reinterpret_cast<uintptr_t>(v) % 16) % 16 / 4));
  if (threadIdx.x < head) top = magnitude(__ldg(v + threadIdx.x));
  const auto* v4 = reinterpret_cast<const float4*>(v + head);
  const int64_t n4 = (n - head) / 4;
#pragma unroll 4
  for (int64_t i = threadIdx.x; i < n4; i += blockDim.x) {
    const float4 f = __ldg(v4 + i);
    top = max(top, max(max(magnitude(f.x), magnitude(f.y)), max(magnitude(f.z), magnitude(f.w))));
  }
  const int64_t tail = head + n4 * 4 + threadIdx.x;
  if (tail < n) top = max(top, magnitude(__ldg(v + tail)));
  return top;
}

// A CTA has one row at a time in registers, 8 values an item and 4 items a
// thread (longer rows are read a second time), and its items' scales with them.
// With wn = ws over the power of two of the largest, |dy * wn| < 2 a.
template <int DT, bool VEC, bool MASK>
__global__ void __launch_bounds__(512) grad_operand_kernel(const GradOperandJob job) {
  constexpr int U = 4;
  __shared__ uint32_t slots[3][32];
  pdl_wait();
  pdl_launch_dependents();
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
       i < job.count_words; i += static_cast<int64_t>(gridDim.x) * blockDim.x)
    job.counts[i] = 0;
  const int64_t items = static_cast<int64_t>(job.KB) * 8;
  const auto* dy = static_cast<const uint16_t*>(job.dy);
  const auto* y = static_cast<const uint16_t*>(job.y);
  // (a power of two of the largest scale in [1, 2))
  const RowPower channel = row_power(__uint_as_float(block_max(top_of(job.ws, job.N), slots[2])));
  const float to_one = channel.rescale * 0x1p-14f, from_one = channel.unscale * 0x1p14f;
  float held_ws[U][8];
  const auto load_ws = [&](int64_t c, float (&ws)[8]) {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      ws[j] = c * 8 + j < job.N ? __ldg(job.ws + c * 8 + j) * to_one : 0.0f;
  };
  const auto load = [&](int64_t m, int64_t c) {
    uint4 v = load_halves<VEC>(dy, m * job.N, c * 8, job.N);
    if constexpr (MASK) {
      const uint4 a = load_halves<VEC>(y, m * job.N, c * 8, job.N);
      v.x &= above_zero<DT>(a.x);
      v.y &= above_zero<DT>(a.y);
      v.z &= above_zero<DT>(a.z);
      v.w &= above_zero<DT>(a.w);
    }
    return v;
  };
  const auto top16 = [&](uint4 v) {
    const uint32_t t = __vmaxu2(__vmaxu2(v.x & 0x7fff7fffu, v.y & 0x7fff7fffu),
                                __vmaxu2(v.z & 0x7fff7fffu, v.w & 0x7fff7fffu));
    return magnitude(half_bits_to_float<DT>(max(t & 0xffffu, t >> 16)));
  };
  const auto put = [&](int64_t m, int64_t c, uint4 v, const float (&ws)[8], float rescale) {
    const uint32_t d[4] = {v.x, v.y, v.z, v.w};
    uint32_t r[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
      r[j] = grad_bits(half_bits_to_float<DT>(d[j] & 0xffffu) * rescale * ws[2 * j]) |
             (static_cast<uint32_t>(
                  grad_bits(half_bits_to_float<DT>(d[j] >> 16) * rescale * ws[2 * j + 1]))
              << 16);
    *reinterpret_cast<uint4*>(job.dst + ((c >> 3) * job.M + m) * 64 + (c & 7) * 8) =
        make_uint4(r[0], r[1], r[2], r[3]);
  };
#pragma unroll
  for (int u = 0; u < U; ++u) load_ws(threadIdx.x + static_cast<int64_t>(u) * blockDim.x, held_ws[u]);
  int turn = 0;
  for (int64_t m = blockIdx.x; m < job.M; m += gridDim.x, turn ^= 1) {
    uint4 held[U];
    uint32_t top = 0;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t c = threadIdx.x + static_cast<int64_t>(u) * blockDim.x;
      held[u] = c < items ? load(m, c) : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) top = max(top, top16(held[u]));
    for (int64_t c = threadIdx.x + static_cast<int64_t>(U) * blockDim.x; c < items; c += blockDim.x)
      top = max(top, top16(load(m, c)));
    // the row's largest between 2^13 and 2^14, times |wn| < 2
    const RowPower row = row_power(2.0f * __uint_as_float(block_max(top, slots[turn])));
    if (threadIdx.x == 0) job.unscale[m] = row.unscale * from_one;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t c = threadIdx.x + static_cast<int64_t>(u) * blockDim.x;
      if (c < items) put(m, c, held[u], held_ws[u], row.rescale);
    }
    for (int64_t c = threadIdx.x + static_cast<int64_t>(U) * blockDim.x; c < items;
         c += blockDim.x) {
      float ws[8];
      load_ws(c, ws);
      put(m, c, load(m, c), ws, row.rescale);
    }
  }
}

// The gated gradient's rows before g and u are known: |u| and |g| are below
//   s[m] * 127 * 128 K * (largest ws) + (largest bias)
// (of typical ones some 7 sqrt(K) times), |act| below |g|, |act'| below
// kSteepest; so with the row's largest |dh| its operand has a bound.
template <int DT, bool VEC_Q, bool VEC_DH>
__global__ void __launch_bounds__(512) gated_grad_front_kernel(const GatedGradFrontJob job) {
  __shared__ uint32_t slots[6][32];
  pdl_wait();
  pdl_launch_dependents();
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
       i < job.count_words; i += static_cast<int64_t>(gridDim.x) * blockDim.x)
    job.counts[i] = 0;
  float top[4];   // of the gate's and the up projection's scales, and of their biases
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float* v = i < 2 ? job.ws : job.bias;
    top[i] = v == nullptr ? 0.0f
                          : __uint_as_float(block_max(top_of(v + (i & 1) * job.N, job.N), slots[i]));
  }
  const float most = 16384.0f * static_cast<float>(job.K);   // |sum| of int8 products
  const auto* dh = static_cast<const uint16_t*>(job.dh);
  const int64_t items = (job.N + 7) / 8, chunks = static_cast<int64_t>(job.KB) * 8;
  int turn = 0;
  for (int64_t m = blockIdx.x; m < job.M; m += gridDim.x, turn ^= 1) {
    uint32_t t = 0;
#pragma unroll 4
    for (int64_t c = threadIdx.x; c < items; c += blockDim.x) {
      const uint4 v = load_halves<VEC_DH>(dh, m * job.N, c * 8, job.N);
      t = __vmaxu2(t, __vmaxu2(__vmaxu2(v.x & 0x7fff7fffu, v.y & 0x7fff7fffu),
                               __vmaxu2(v.z & 0x7fff7fffu, v.w & 0x7fff7fffu)));
    }
#pragma unroll 2
    for (int64_t c = threadIdx.x; c < chunks; c += blockDim.x) {
      const int8_t* src = job.q + m * job.K + c * 8;
      uint2 w = make_uint2(0, 0);
      if constexpr (VEC_Q) {
        if (c * 8 < job.K) w = *reinterpret_cast<const uint2*>(src);
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (c * 8 + j < job.K)
            (j < 4 ? w.x : w.y) |= static_cast<uint32_t>(static_cast<uint8_t>(src[j])) << (8 * (j & 3));
      }
      *reinterpret_cast<uint4*>(job.operand + ((c >> 3) * job.M + m) * 64 + (c & 7) * 8) =
          token_f16x8(w);
    }
    const uint32_t most_dh =
        block_max(magnitude(half_bits_to_float<DT>(max(t & 0xffffu, t >> 16))), slots[4 + turn]);
    if (threadIdx.x == 0) {
      const float acc = fabsf(job.scales[m]) * most;
      const float g = fmaf(acc, top[0], top[2]), u = fmaf(acc, top[1], top[3]);
      const RowPower row = row_power(__uint_as_float(most_dh) * kSteepest * fmaxf(u * top[0], g * top[1]));
      job.rescale[m] = row.rescale;
      job.unscale[m] = row.unscale;
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

template <typename F>
cudaError_t by_half(q8_dtype dt, bool vec, F&& f) {
  const auto with = [&](auto t) { return vec ? f(t, std::true_type()) : f(t, std::false_type()); };
  return dt == Q8_F16 ? with(std::integral_constant<int, Q8_F16>())
                      : with(std::integral_constant<int, Q8_BF16>());
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
  const int64_t items = static_cast<int64_t>(job.KB) * 8;
  const int64_t each = job.M <= 2 * device_sm_count() ? 1 : 4;
  const int threads = static_cast<int>(
      std::min<int64_t>(512, std::max<int64_t>(64, round_up((items + each - 1) / each, 32))));
  const int grid = static_cast<int>(
      std::min<int64_t>(job.M, static_cast<int64_t>(device_sm_count()) * (1024 / threads)));
  const auto go = [&](auto t, auto v) {
    constexpr int DT = decltype(t)::value;
    constexpr bool VEC = decltype(v)::value;
    return job.y != nullptr ? launch_pdl(grad_operand_kernel<DT, VEC, true>, grid, threads, 0, s, job)
                            : launch_pdl(grad_operand_kernel<DT, VEC, false>, grid, threads, 0, s, job);
  };
  return by_half(dtype, vec, go);
}

cudaError_t launch_gated_grad_front(const GatedGradFrontJob& job, q8_dtype dtype, cudaStream_t s) {
  const bool vec_dh = job.N % 8 == 0 && on16(job.dh);
  const bool vec_q = job.K % 8 == 0 && reinterpret_cast<uintptr_t>(job.q) % 8 == 0;
  const int grid = static_cast<int>(std::min<int64_t>(job.M, device_sm_count() * 2));
  return by_half(dtype, vec_dh, [&](auto t, auto v) {
    constexpr int DT = decltype(t)::value;
    constexpr bool VEC = decltype(v)::value;
    return vec_q ? launch_pdl(gated_grad_front_kernel<DT, true, VEC>, grid, 512, 0, s, job)
                 : launch_pdl(gated_grad_front_kernel<DT, false, VEC>, grid, 512, 0, s, job);
  });
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
