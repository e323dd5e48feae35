// token_rows.cu -- the products of few rows with a scale for each token, and the
// gated pair of them: one launch that quantizes the rows and reads each weight
// once, as fast as memory gives them.
//
//   acc[m, n] = sum_k q[m, k] w[n, k]   exact in int32
//   v = ((float)acc * s[m]) * ws[n] + b[n];   gated: act(v_gate) * v_up
//
// Up to 8 rows a weight's 1 byte costs more than its 2 to 16 operations, so
// bytes in flight count.  A CTA of 16 warps takes units of 16 packed rows (16
// channels, or 8 of both halves of a gated pair); the warps share a unit's
// inputs, four 16-byte loads ahead each (32 KB a CTA, two CTAs an SM; 44 bytes
// a nanosecond and SM at the copy rate with 800 ns of latency want 35).  They run
// on across units, and the first ones are asked for before the kernel before
// this one is done (a packed weight is written at load time).  Rows x inputs x
// outputs, in a run of calls: 1 x 11008 x 4096 10.7 us (floor 6.8), the gated pair
// 1 x 4096 x 11008 17.7 us (13.6); 1 x 1024 x 1024, which is all latency, 2.8 us.
// Code that runs once costs more to fetch than to execute: with eight loads ahead
// those were 10.5, 17.9 and 3.1, with a row's first 4 items held instead of 2 11.0,
// 18.4 and 3.1.
//   One or two rows: four products a dp4a, straight from the registers that the
// loads fill; the rows' int8 come from shared memory, 16 bytes that half a warp
// shares.  That is a load from there for each row and load of weights, of which an
// SM can do two, so three to eight rows go through m16n8k16 MMAs, f16 in and f32
// out: the packed 16-byte chunks are a thread's fragments as they lie (the order
// of a sum's terms is free, so thread t of four takes inputs 16 t to 16 t + 15 of
// a k-block), turned into f16 by a byte permute and half a subtraction a value,
// and rows are the MMA's 8 columns.  Products are at most 2^14 and a chunk of 8 k-blocks adds
// 512 of them, so its f32 sums are exact integers; they are then added up in
// int32, across warps too, so the order does not matter.
//   Every CTA quantizes all rows for itself (one row of 4096 is 8 KB from L2,
// beside 65 KB of weights for each unit): that saves a launch, and the scales
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
constexpr int kAhead = 4;         // 16-byte loads in flight a thread
constexpr int kExactBlocks = 8;   // k-blocks of one exact f32 chunk

__device__ __forceinline__ uint4 load_weights(const uint4* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                        uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

struct RowsShared {
  uint32_t top[kRowWarps];   // each warp's
  float scale[kFewRows];
};

// All rows as int8 in shared memory, zeros from K on, biased by 128 under BIAS;
// their scales, and for the first CTA what the caller wants of both.  A warp has
// one row, alone or with others while there are more warps than rows, and keeps
// the first items of its share in registers while the row's scale is found.
template <int DT, bool VEC, bool BIAS>
__device__ __forceinline__ void stage_rows(const TokenRowsJob& job, RowsShared& sh, uint8_t* rows) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int M = static_cast<int>(job.M);
  const int each = kRowWarps / M, m = warp / each;   // warps a row
  const int part = (warp - m * each) * 32 + lane, step = each * 32;
  const int padded = job.KB * 64;
  const bool mine = m < M;
  constexpr uint32_t kFlip = BIAS ? 0x80808080u : 0;
  const int64_t base = static_cast<int64_t>(mine ? m : 0) * job.K;
  uint8_t* dst = rows + (mine ? m : 0) * job.stride;
  if constexpr (DT == Q8_I8) {
    if (threadIdx.x < M) sh.scale[threadIdx.x] = job.scales[threadIdx.x];
    const int8_t* src = static_cast<const int8_t*>(job.x) + base;
    if (mine) {
      if constexpr (VEC) {
#pragma unroll 4
        for (int c = part; c < padded / 16; c += step) {
          uint4 v = c * 16 < job.K ? *reinterpret_cast<const uint4*>(src + c * 16)
                                   : make_uint4(0, 0, 0, 0);
          v.x ^= kFlip;
          v.y ^= kFlip;
          v.z ^= kFlip;
          v.w ^= kFlip;
          *reinterpret_cast<uint4*>(dst + c * 16) = v;
        }
      } else {
        const int8_t* all = static_cast<const int8_t*>(job.x);
#pragma unroll 4
        for (int c = part; c < padded / 8; c += step) {
          uint2 v = load_int8x8<false>(all, base, static_cast<int64_t>(c) * 8, job.K, all + M * job.K);
          v.x ^= kFlip;
          v.y ^= kFlip;
          *reinterpret_cast<uint2*>(dst + c * 8) = v;
        }
      }
    }
  } else {
    using Item = TokenItem<DT, VEC>;
    constexpr int U = DT == Q8_F32 || !VEC ? 1 : 2;
    // items of 8 up to the end of the last k-block, by whole warps
    const int items = mine ? padded / 8 : 0;
    const int64_t bytes = mine ? job.K * static_cast<int64_t>(sizeof(FloatOf<DT>)) : 0;
    const RowBytes row = row_bytes<FloatOf<DT>>(job.x, M, job.K, mine ? m : 0);
    Item held[U];
    uint32_t top = 0;
#pragma unroll
    for (int u = 0; u < U; ++u) held[u].load(row, part + u * step, bytes);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      held[u].settle(row, part + u * step, bytes);
      top = max(top, held[u].top());
    }
#pragma unroll 1
    for (int c = part + U * step; c < items; c += step) {
      Item it;
      it.load(row, c, bytes);
      it.settle(row, c, bytes);
      top = max(top, it.top());
    }
    top = __reduce_max_sync(0xffffffffu, top);
    if (lane == 0) sh.top[warp] = top;
    __syncthreads();
    top = __reduce_max_sync(0xffffffffu, mine && lane < each ? sh.top[m * each + lane] : 0u);
    const TokenScale sc = token_scale(top);
    if (mine && part == 0) {
      sh.scale[m] = sc.scale;
      if (blockIdx.x == 0 && job.scales != nullptr) job.scales[m] = sc.scale;
    }
    const auto put = [&](const Item& it, int c) {
      uint2 q = it.quantize(sc.inv);   // (zeros past K)
      if (blockIdx.x == 0 && job.q != nullptr)
        store_bytes_any(job.q + base + c * 8, q,
                        static_cast<int>(min(int64_t{8}, job.K - static_cast<int64_t>(c) * 8)));
      if (c < items) {
        q.x ^= kFlip;
        q.y ^= kFlip;
        *reinterpret_cast<uint2*>(dst + c * 8) = q;
      }
    };
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (part - lane + u * step < items) put(held[u], part + u * step);
#pragma unroll 1
    for (int c = part + U * step; c - lane < items; c += step) {
      Item it;
      it.load(row, c, bytes);
      it.settle(row, c, bytes);
      put(it, c);
    }
  }
  __syncthreads();
}

template <bool BIAS>
__device__ __forceinline__ void stage_rows_by_type(const TokenRowsJob& job, RowsShared& sh,
                                                   uint8_t* rows) {
  switch (job.x_dtype * 2 + job.vec) {
    case Q8_I8 * 2: stage_rows<Q8_I8, false, BIAS>(job, sh, rows); break;
    case Q8_I8 * 2 + 1: stage_rows<Q8_I8, true, BIAS>(job, sh, rows); break;
    case Q8_F32 * 2: stage_rows<Q8_F32, false, BIAS>(job, sh, rows); break;
    case Q8_F32 * 2 + 1: stage_rows<Q8_F32, true, BIAS>(job, sh, rows); break;
    case Q8_F16 * 2: stage_rows<Q8_F16, false, BIAS>(job, sh, rows); break;
    case Q8_F16 * 2 + 1: stage_rows<Q8_F16, true, BIAS>(job, sh, rows); break;
    case Q8_BF16 * 2: stage_rows<Q8_BF16, false, BIAS>(job, sh, rows); break;
    default: stage_rows<Q8_BF16, true, BIAS>(job, sh, rows); break;
  }
}

// MT: rows that the kernel has sums for, M at least; up to 2 by dp4a, else MMAs.
template <int MT, bool GATED>
__global__ void __launch_bounds__(kRowThreads, 2) token_rows_kernel(const TokenRowsJob job) {
  constexpr bool kMma = MT > 2;
  static_assert(!kMma || MT == 8, "an MMA's columns");
  constexpr int kLoads = kMma ? 2 : 1;               // of a thread to a piece
  constexpr int kDeep = kAhead / kLoads;             // pieces on their way
  extern __shared__ __align__(16) uint8_t dyn[];
  __shared__ RowsShared sh;
  // two units' sums, so that one barrier a unit keeps them apart
  auto* parts = reinterpret_cast<int32_t(*)[kRowWarps][MT][16]>(dyn);
  uint8_t* rows = dyn + sizeof(int32_t) * 2 * kRowWarps * MT * 16;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, r = lane & 15, half = lane >> 4;
  const int g = lane >> 2, t = lane & 3;
  const int M = static_cast<int>(job.M);
  // pieces of 32 inputs, or of 64 for the MMAs
  const int pieces = kMma ? job.KB : job.KB * 2;
  const int rounds = (pieces + kRowWarps * kDeep - 1) / (kRowWarps * kDeep);

  const auto load = [&](uint4 (&a)[kLoads], int unit, int piece) {
    if (unit < job.units && piece < pieces) {
      const uint4* w = reinterpret_cast<const uint4*>(job.w) +
                       static_cast<int64_t>(unit >> 3) * job.KB * 512;
      const int row = GATED ? ((unit & 6) << 4) + ((unit & 1) << 3) : (unit & 7) << 4;
      if constexpr (kMma) {
        w += piece * 512 + t * 128 + row + g;
        a[0] = load_weights(w);
        a[kLoads - 1] = load_weights(w + (GATED ? 16 : 8));
      } else {
        a[0] = load_weights(w + piece * 256 + half * 128 + row + (r & 7) +
                            (GATED ? (r & 8) << 1 : r & 8));
      }
    }
  };
  uint4 a[kDeep][kLoads];
#pragma unroll
  for (int s = 0; s < kDeep; ++s) load(a[s], blockIdx.x, warp + s * kRowWarps);
  pdl_wait();
  pdl_launch_dependents();
  stage_rows_by_type<kMma>(job, sh, rows);

  // the first warps finish two rows each
  const int m = warp * 2 + half;
  const bool up = GATED && (r & 8);
  const float scale = sh.scale[min(m, M - 1)];
  int turn = 0;
  for (int unit = blockIdx.x; unit < job.units; unit += gridDim.x, turn ^= 1) {
    const int n = GATED ? unit * 8 + (r & 7) : unit * 16 + r;
    const bool in = n < job.N && m < M;
    const int64_t en = (up ? job.N : 0) + n;
    float ws = 0.0f, bias = 0.0f;   // on their way early
    if (in) {
      ws = __ldg(job.ws + en);
      if (job.bias != nullptr) bias = __ldg(job.bias + en);
    }
    const auto ahead = [&](int round, int s) {
      // the piece kDeep places on, in the next unit after this one's last
      const bool more = round + 1 < rounds;
      load(a[s], more ? unit : unit + gridDim.x,
           warp + ((more ? (round + 1) * kDeep : 0) + s) * kRowWarps);
    };
    if constexpr (kMma) {
      const __half2 minus = __halves2half2(__ushort_as_half(0x6480), __ushort_as_half(0x6480));
      float acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
      int32_t sum[4] = {0, 0, 0, 0};
      const auto drain = [&]() {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          sum[j] += __float2int_rn(acc[j]);
          acc[j] = 0.0f;
        }
      };
      for (int round = 0; round < rounds; ++round) {
#pragma unroll
        for (int s = 0; s < kDeep; ++s) {
          const int piece = warp + (round * kDeep + s) * kRowWarps;
          if (piece < pieces) {
            const uint4 &lo = a[s][0], &hi = a[s][kLoads - 1];
            uint4 v = make_uint4(0x80808080u, 0x80808080u, 0x80808080u, 0x80808080u);
            if (g < M) v = *reinterpret_cast<const uint4*>(rows + g * job.stride + piece * 64 + t * 16);
            const auto four = [&](uint32_t wlo, uint32_t whi, uint32_t x) {
              mma_f16(acc, biased_to_f16x2(wlo, 0x4140, minus), biased_to_f16x2(whi, 0x4140, minus),
                      biased_to_f16x2(wlo, 0x4342, minus), biased_to_f16x2(whi, 0x4342, minus),
                      biased_to_f16x2(x, 0x4140, minus), biased_to_f16x2(x, 0x4342, minus));
            };
            four(lo.x, hi.x, v.x);
            four(lo.y, hi.y, v.y);
            four(lo.z, hi.z, v.z);
            four(lo.w, hi.w, v.w);
          }
          ahead(round, s);
        }
        if ((round + 1) % (kExactBlocks / kDeep) == 0) drain();
      }
      drain();
#pragma unroll
      for (int j = 0; j < 4; ++j) parts[turn][warp][2 * t + (j & 1)][g + (j >> 1) * 8] = sum[j];
    } else {
      int32_t acc[MT];
#pragma unroll
      for (int i = 0; i < MT; ++i) acc[i] = 0;
      for (int round = 0; round < rounds; ++round) {
#pragma unroll
        for (int s = 0; s < kDeep; ++s) {
          const int piece = warp + (round * kDeep + s) * kRowWarps;
          if (piece < pieces) {
            const uint8_t* x = rows + piece * 32 + half * 16;
#pragma unroll
            for (int i = 0; i < MT; ++i) {
              const uint4 q = *reinterpret_cast<const uint4*>(x + min(i, M - 1) * job.stride);
              acc[i] = __dp4a(static_cast<int>(a[s][0].x ^ 0x80808080u), static_cast<int>(q.x), acc[i]);
              acc[i] = __dp4a(static_cast<int>(a[s][0].y ^ 0x80808080u), static_cast<int>(q.y), acc[i]);
              acc[i] = __dp4a(static_cast<int>(a[s][0].z ^ 0x80808080u), static_cast<int>(q.z), acc[i]);
              acc[i] = __dp4a(static_cast<int>(a[s][0].w ^ 0x80808080u), static_cast<int>(q.w), acc[i]);
            }
          }
          ahead(round, s);
        }
      }
#pragma unroll
      for (int i = 0; i < MT; ++i) {
        acc[i] += __shfl_xor_sync(0xffffffffu, acc[i], 16);
        if (half == 0) parts[turn][warp][i][r] = acc[i];
      }
    }
    __syncthreads();
    if (warp * 2 < M) {
      int32_t total = 0;
#pragma unroll
      for (int w = 0; w < kRowWarps; ++w) total += parts[turn][w][min(m, M - 1)][r];
      float v = token_value(total, scale, ws, bias);
      if constexpr (GATED) {
        const float other = __shfl_xor_sync(0xffffffffu, v, 8);
        float slope;
        if (!up)
          v = (job.out_dtype == Q8_F32 ? activate<false, true>(v, job.act, slope)
                                       : activate<false, false>(v, job.act, slope)) *
              other;
      } else if (job.act == kActRelu) {
        v = max_nan(v, 0.0f);
      }
      if (in && !up) {
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
constexpr size_t kTwoShared = 110 * 1024;    // of each of two CTAs

int rows_of(int64_t M) { return M <= 2 ? static_cast<int>(M) : 8; }
size_t rows_shared(int64_t M, int64_t K) {
  return static_cast<size_t>(2 * kRowWarps * 16 * 4) * rows_of(M) +
         static_cast<size_t>(M) * token_rows_stride(K);
}

template <int MT, bool GATED>
cudaError_t launch_rows(const TokenRowsJob& job, cudaStream_t s) {
  auto kernel = token_rows_kernel<MT, GATED>;
  static DeviceOnce once;
  cudaError_t e = once.run([&] {
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                static_cast<int>(kMostShared));
  });
  if (e != cudaSuccess) return e;
  const size_t shared = rows_shared(job.M, job.K);
  const int grid = std::min(job.units, device_sm_count() * (shared <= kTwoShared ? 2 : 1));
  return launch_pdl(kernel, grid, kRowThreads, shared, s, job);
}

template <bool GATED>
cudaError_t launch_by_rows(const TokenRowsJob& job, cudaStream_t s) {
  switch (rows_of(job.M)) {
    case 1: return launch_rows<1, GATED>(job, s);
    case 2: return launch_rows<2, GATED>(job, s);
    default: return launch_rows<8, GATED>(job, s);
  }
}

}  // namespace

// Every CTA quantizes all rows, so many long ones are left to the other kernel
// (rows_internal.h), whose time does not depend on a few rows.  Measured, here
// against there, rows x inputs x outputs, bf16: 1 x 11008 x 4096 10.2 us, 16.7;
// 1 x 28672 22.5, 28.0; 2 x 28672 25.6, 27.8; 4 x 4096 9.7, 12.1; 8 x 4096 11.3,
// 12.3; 4 x 8192 14.6, 14.9; 8 x 11008 24.1, 16.7 (all x 4096); and 16 x 2048 x
// 11008 16.5, 11.9.
// int8 rows are only copied, and a product by one weight gains up to twice the
// values: 8 x 4160 8.2 us, 11.0; 4 x 11008 13.5, 15.6; 8 x 8192 11.6, 13.8 (all
// x 4096); 6 x 6000 x 8000 15.2, 15.9; 8 x 11008 15.2, 15.7.  By a gated weight
// they do not: 6 x 6000 x 8000 25.5, 22.1; 4 x 11008 x 4096 23.9, 23.2.
bool token_rows_fit(int64_t M, int64_t K, bool copied) {
  return M >= 1 && M <= kFewRows && K <= (1 << 20) &&
         (M <= 2 || M * K <= (copied ? 65536 : 32768)) && rows_shared(M, K) <= kMostShared;
}

cudaError_t launch_token_rows(TokenRowsJob job, bool gated, cudaStream_t s) {
  job.KB = static_cast<int>((job.K + 63) / 64);
  job.stride = static_cast<int>(token_rows_stride(job.K));
  job.units = static_cast<int>(gated ? (job.N + 7) / 8 : (job.N + 15) / 16);
  // (VEC's items of 8 float values, or 16 int8 ones, are whole)
  job.vec = job.K % (job.x_dtype == Q8_I8 ? 16 : 8) == 0 && reinterpret_cast<uintptr_t>(job.x) % 16 == 0;
  return gated ? launch_by_rows<true>(job, s) : launch_by_rows<false>(job, s);
}

}  // namespace q8
