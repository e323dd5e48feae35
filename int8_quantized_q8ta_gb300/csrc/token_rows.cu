// token_rows.cu -- the products of few rows with a scale for each token, and the
// gated pair of them: one launch that quantizes the rows and reads each weight
// once, as fast as memory gives them.
//
//   acc[m, n] = sum_k q[m, k] w[n, k]   exact in int32
//   v = ((float)acc * s[m]) * ws[n] + b[n];   gated: act(v_gate) * v_up
//
// Up to 16 rows a weight's 1 byte costs more than its 2 to 32 operations, so
// bytes in flight count.  A CTA of 16 warps takes units of 32 packed rows (32
// channels, or 16 of both halves of a gated pair); its warps share a unit's
// k-blocks, and each has its next two k-blocks' weights on their way in
// registers (4 KB a warp, 64 KB an SM; 44 bytes a nanosecond and SM at the copy
// rate with 800 ns of latency want 35).  They run on across units, and the first
// ones are asked for before the kernel before this one is done (a packed weight
// is written at load time).
//   Weights go from memory to registers to m16n8k16 MMAs, f16 in and f32 out:
// packed 16-byte chunks are a thread's fragments as they lie (the order of a
// sum's terms is free, so thread t of four takes inputs 16 t to 16 t + 15 of a
// k-block), turned into f16 by a byte permute and half a subtraction a value.
// Rows are the MMAs' 8 columns; int8, biased alike, in shared memory.  Products
// are at most 2^14 and a chunk of 8 k-blocks adds 512 of them, so its f32 sums
// are exact integers; they are then added up in int32, across warps too, so the
// order does not matter.
//   Every CTA quantizes all rows for itself (one row of 4096 is 8 KB from L2,
// beside 131 KB of weights for each unit): that saves a launch, and the scales
// and int8 rows that the caller wants are written by the first CTA.
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "token_device.cuh"
#include "token_internal.h"

namespace q8 {

namespace {

constexpr int kRowWarps = 16, kRowThreads = kRowWarps * 32;
constexpr int kAhead = 2;         // k-blocks of weights in flight a warp
constexpr int kExactBlocks = 8;   // k-blocks of one exact f32 chunk

__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                        uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

struct RowsShared {
  uint32_t top[kFewRows];
  float scale[kFewRows];
};

// All rows as biased int8 in shared memory, zeros (0x80) from K on; their
// scales, and for the first CTA what the caller wants of both.  Warps share the
// rows: a few warps a row while there are more warps than rows, else rows in
// turn.
template <int DT, bool VEC>
__device__ __forceinline__ void stage_rows(const TokenRowsJob& job, RowsShared& sh, uint8_t* rows) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int M = static_cast<int>(job.M);
  const int each = max(1, kRowWarps / M);             // warps a row
  const int first = warp / each, part = (warp % each) * 32 + lane, step = each * 32;
  const int row_step = max(1, kRowWarps / each);
  const int padded = job.KB * 64;
  if constexpr (DT == Q8_I8) {
    if (threadIdx.x < M) sh.scale[threadIdx.x] = job.scales[threadIdx.x];
    const auto* x = static_cast<const int8_t*>(job.x);
    for (int m = first; m < M; m += row_step) {
      const int8_t* src = x + static_cast<int64_t>(m) * job.K;
      uint8_t* dst = rows + m * job.stride;
      if constexpr (VEC) {
#pragma unroll 4
        for (int c = part; c < padded / 16; c += step) {
          uint4 v = c * 16 < job.K ? *reinterpret_cast<const uint4*>(src + c * 16)
                                   : make_uint4(0, 0, 0, 0);
          v.x ^= 0x80808080u;
          v.y ^= 0x80808080u;
          v.z ^= 0x80808080u;
          v.w ^= 0x80808080u;
          *reinterpret_cast<uint4*>(dst + c * 16) = v;
        }
      } else {
#pragma unroll 4
        for (int k = part; k < padded; k += step)
          dst[k] = k < job.K ? static_cast<uint8_t>(src[k]) ^ 0x80 : 0x80;
      }
    }
  } else {
    using Item = TokenItem<DT, VEC>;
    constexpr int W = Item::kWidth;
    const int items = static_cast<int>(job.K) / W;
    if (threadIdx.x < kFewRows) sh.top[threadIdx.x] = 0;
    __syncthreads();
    for (int m = first; m < M; m += row_step) {
      const int64_t base = static_cast<int64_t>(m) * job.K;
      uint32_t top = 0;
#pragma unroll 4
      for (int c = part; c < items; c += step) {
        Item it;
        it.load(job.x, base + c * W);
        top = max(top, it.top());
      }
      top = __reduce_max_sync(0xffffffffu, top);
      if (lane == 0) atomicMax(&sh.top[m], top);
    }
    __syncthreads();
    if (threadIdx.x < M) {
      const float s = token_scale(sh.top[threadIdx.x]).scale;
      sh.scale[threadIdx.x] = s;
      if (blockIdx.x == 0 && job.scales != nullptr) job.scales[threadIdx.x] = s;
    }
    for (int m = first; m < M; m += row_step) {
      const int64_t base = static_cast<int64_t>(m) * job.K;
      const float inv = token_scale(sh.top[m]).inv;
      uint8_t* dst = rows + m * job.stride;
#pragma unroll 4
      for (int c = part; c < items; c += step) {
        Item it;
        it.load(job.x, base + c * W);
        if constexpr (VEC) {
          uint2 q = it.quantize(inv);
          if (blockIdx.x == 0 && job.q != nullptr) {
            // (the caller's rows may lie on any byte)
            int8_t* to = job.q + base + c * 8;
#pragma unroll
            for (int j = 0; j < 8; ++j)
              to[j] = static_cast<int8_t>((j < 4 ? q.x : q.y) >> (8 * (j & 3)));
          }
          q.x ^= 0x80808080u;
          q.y ^= 0x80808080u;
          *reinterpret_cast<uint2*>(dst + c * 8) = q;
        } else {
          const int8_t q = it.quantize(inv);
          if (blockIdx.x == 0 && job.q != nullptr) job.q[base + c] = q;
          dst[c] = static_cast<uint8_t>(q) ^ 0x80;
        }
      }
      for (int k = static_cast<int>(job.K) + part; k < padded; k += step) dst[k] = 0x80;
    }
  }
  __syncthreads();
}

template <int NT, bool GATED>
__global__ void __launch_bounds__(kRowThreads, 1) token_rows_kernel(const TokenRowsJob job) {
  constexpr int kCols = 8 * NT + 1;   // words of a partial row (odd: no bank twice)
  extern __shared__ __align__(16) uint8_t dyn[];
  __shared__ RowsShared sh;
  auto* parts = reinterpret_cast<int32_t*>(dyn);                    // [warps][32][kCols]
  uint8_t* rows = dyn + kRowWarps * 32 * kCols * 4;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int M = static_cast<int>(job.M), KB = job.KB;
  const int rounds = (KB + kRowWarps * kAhead - 1) / (kRowWarps * kAhead);

  // this thread's four 16-byte chunks of a unit's k-block: rows g, g + 8, ...
  const auto load = [&](uint4 (&a)[4], int unit, int kb) {
    if (unit < job.units && kb < KB) {
      const auto* w = reinterpret_cast<const uint4*>(
          job.w + (static_cast<int64_t>(unit >> 2) * KB + kb) * 8192 + (unit & 3) * 512 + t * 2048 +
          g * 16);
#pragma unroll
      for (int i = 0; i < 4; ++i) a[i] = __ldcs(w + i * 8);
    }
  };
  uint4 a[kAhead][4];
#pragma unroll
  for (int s = 0; s < kAhead; ++s) load(a[s], blockIdx.x, warp + s * kRowWarps);
  pdl_wait();
  pdl_launch_dependents();
  switch (job.x_dtype) {
    case Q8_I8: job.vec ? stage_rows<Q8_I8, true>(job, sh, rows) : stage_rows<Q8_I8, false>(job, sh, rows); break;
    case Q8_F32: job.vec ? stage_rows<Q8_F32, true>(job, sh, rows) : stage_rows<Q8_F32, false>(job, sh, rows); break;
    case Q8_F16: job.vec ? stage_rows<Q8_F16, true>(job, sh, rows) : stage_rows<Q8_F16, false>(job, sh, rows); break;
    default: job.vec ? stage_rows<Q8_BF16, true>(job, sh, rows) : stage_rows<Q8_BF16, false>(job, sh, rows); break;
  }

  const __half2 minus = __halves2half2(__ushort_as_half(0x6480), __ushort_as_half(0x6480));
  for (int unit = blockIdx.x; unit < job.units; unit += gridDim.x) {
    // this thread's channel of the unit's outputs, its scales on their way early
    const int n = GATED ? unit * 16 + (threadIdx.x & 15) : unit * 32 + (threadIdx.x & 31);
    const bool in = n < job.N;
    float ws[2] = {0.0f, 0.0f}, bias[2] = {0.0f, 0.0f};
#pragma unroll
    for (int h = 0; h < (GATED ? 2 : 1); ++h)
      if (in) {
        ws[h] = __ldg(job.ws + static_cast<int64_t>(h) * job.N + n);
        if (job.bias != nullptr) bias[h] = __ldg(job.bias + static_cast<int64_t>(h) * job.N + n);
      }
    float acc[NT][2][4];
    int32_t sum[NT][2][4];
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          acc[i][h][j] = 0.0f;
          sum[i][h][j] = 0;
        }
    const auto drain = [&]() {
#pragma unroll
      for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            sum[i][h][j] += __float2int_rn(acc[i][h][j]);
            acc[i][h][j] = 0.0f;
          }
    };
    for (int r = 0; r < rounds; ++r) {
#pragma unroll
      for (int s = 0; s < kAhead; ++s) {
        const int kb = warp + (r * kAhead + s) * kRowWarps;
        if (kb < KB) {
          uint32_t b[NT][8];
#pragma unroll
          for (int i = 0; i < NT; ++i) {
            const int m = i * 8 + g;
            uint4 v = make_uint4(0x80808080u, 0x80808080u, 0x80808080u, 0x80808080u);
            if (m < M) v = *reinterpret_cast<const uint4*>(rows + m * job.stride + kb * 64 + t * 16);
            const uint32_t q[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              b[i][2 * j] = biased_to_f16x2(q[j], 0x4140, minus);
              b[i][2 * j + 1] = biased_to_f16x2(q[j], 0x4342, minus);
            }
          }
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint32_t lo[4] = {a[s][2 * h].x, a[s][2 * h].y, a[s][2 * h].z, a[s][2 * h].w};
            const uint32_t hi[4] = {a[s][2 * h + 1].x, a[s][2 * h + 1].y, a[s][2 * h + 1].z,
                                    a[s][2 * h + 1].w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const uint32_t a0 = biased_to_f16x2(lo[j], 0x4140, minus);
              const uint32_t a1 = biased_to_f16x2(hi[j], 0x4140, minus);
              const uint32_t a2 = biased_to_f16x2(lo[j], 0x4342, minus);
              const uint32_t a3 = biased_to_f16x2(hi[j], 0x4342, minus);
#pragma unroll
              for (int i = 0; i < NT; ++i)
                mma_f16(acc[i][h], a0, a1, a2, a3, b[i][2 * j], b[i][2 * j + 1]);
            }
          }
        }
        // the k-block kAhead places on, in the next unit after this one's last
        const bool more = r + 1 < rounds;
        load(a[s], more ? unit : unit + gridDim.x,
             warp + ((more ? (r + 1) * kAhead : 0) + s) * kRowWarps);
      }
      if ((r + 1) % (kExactBlocks / kAhead) == 0) drain();
    }
    drain();
    __syncthreads();   // the unit before has been read
    int32_t* mine = parts + warp * 32 * kCols;
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int j = 0; j < 4; ++j)
          mine[(h * 16 + (j >> 1) * 8 + g) * kCols + i * 8 + 2 * t + (j & 1)] = sum[i][h][j];
    __syncthreads();
    constexpr int kChannels = GATED ? 16 : 32;
    for (int i = threadIdx.x; i < kChannels * M; i += kRowThreads) {
      const int row = i % kChannels, m = i / kChannels;
      int32_t total[2] = {0, 0};
#pragma unroll
      for (int w = 0; w < kRowWarps; ++w)
#pragma unroll
        for (int h = 0; h < (GATED ? 2 : 1); ++h)
          total[h] += parts[(w * 32 + h * 16 + row) * kCols + m];
      if (in) {
        float v = token_value(total[0], sh.scale[m], ws[0], bias[0]);
        if constexpr (GATED) {
          float slope;
          v = activate<false>(v, job.act, slope) * token_value(total[1], sh.scale[m], ws[1], bias[1]);
        } else if (job.act == kActRelu) {
          v = max_nan(v, 0.0f);
        }
        const int64_t at = static_cast<int64_t>(m) * job.N + n;
        switch (job.out_dtype) {
          case Q8_F32: store_one<Q8_F32>(job.out, at, v); break;
          case Q8_F16: store_one<Q8_F16>(job.out, at, v); break;
          default: store_one<Q8_BF16>(job.out, at, v); break;
        }
      }
    }
  }
}

constexpr size_t kMostShared = 220 * 1024;   // beside it the scales

size_t rows_shared(int64_t M, int64_t K) {
  const int nt = M <= 8 ? 1 : 2;
  return static_cast<size_t>(kRowWarps) * 32 * (8 * nt + 1) * 4 + static_cast<size_t>(M) * token_rows_stride(K);
}

template <int NT, bool GATED>
cudaError_t launch_rows(const TokenRowsJob& job, cudaStream_t s) {
  auto kernel = token_rows_kernel<NT, GATED>;
  static DeviceOnce once;
  cudaError_t e = once.run([&] {
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                static_cast<int>(kMostShared));
  });
  if (e != cudaSuccess) return e;
  const int grid = std::min(job.units, device_sm_count());
  return launch_pdl(kernel, grid, kRowThreads, rows_shared(job.M, job.K), s, job);
}

}  // namespace

bool token_rows_fit(int64_t M, int64_t K) {
  return M >= 1 && M <= kFewRows && K <= (1 << 20) && rows_shared(M, K) <= kMostShared;
}

cudaError_t launch_token_rows(TokenRowsJob job, bool gated, cudaStream_t s) {
  job.KB = static_cast<int>((job.K + 63) / 64);
  job.stride = static_cast<int>(token_rows_stride(job.K));
  const int64_t rows = gated ? gated_rows(job.N) : job.N;
  job.units = static_cast<int>((rows + 31) / 32);
  const int64_t bytes = dtype_bytes(job.x_dtype), wide = job.x_dtype == Q8_I8 ? 16 : 8;
  job.vec = job.K % wide == 0 && reinterpret_cast<uintptr_t>(job.x) % 16 == 0 &&
            job.K * bytes % 16 == 0;
  if (job.M <= 8) return gated ? launch_rows<1, true>(job, s) : launch_rows<1, false>(job, s);
  return gated ? launch_rows<2, true>(job, s) : launch_rows<2, false>(job, s);
}

}  // namespace q8
