// tile_prep.cu -- what the grouped int8 contraction (tile_gemm.cu) reads:
// load-time packing of weights and adapters, the token operand, and for
// adapters the rows' low-rank products h and each tile's list of adapters.
#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>
#include <type_traits>

#include "row_split.h"
#include "rows_internal.h"
#include "tile_device.cuh"
#include "token_device.cuh"

namespace q8 {

namespace cg = cooperative_groups;

namespace {

int blocks_for(int64_t items) {
  return static_cast<int>(std::max<int64_t>(
      1, std::min<int64_t>((items + 255) / 256, static_cast<int64_t>(device_sm_count()) * 8)));
}

// One 16-byte chunk (a row's 16 inputs) per item; once, at load time (64 weights
// of 4096 x 4096 0.89 ms, 2.4 TB/s).
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
    uint2 lo = make_uint2(0, 0), hi = lo;
    if (n < N) {   // (whole words wherever the row begins: 11008 x 4096 27 us, by bytes 152)
      const int64_t at = (e * N + n) * K;
      lo = load_int8x8<false>(w, at, k0, K, w + E * N * K);
      hi = load_int8x8<false>(w, at, k0 + 8, K, w + E * N * K);
    }
    dst[i] = make_uint4(lo.x ^ 0x80808080u, lo.y ^ 0x80808080u, hi.x ^ 0x80808080u,
                        hi.y ^ 0x80808080u);
  }
}

// The largest sum of |w| over a row's 64 inputs of one k-block, from packed tiles:
// a thread a row of a tile, four chunks of 16.
__global__ void __launch_bounds__(256) tile_weight_bound_kernel(const uint4* __restrict__ packed,
                                                                int64_t tiles, int32_t* bound) {
  pdl_wait();
  uint32_t best = 0;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; i < tiles * 128;
       i += static_cast<int64_t>(gridDim.x) * blockDim.x) {
    const uint4* row = packed + (i >> 7) * 512 + (i & 127);
    uint4 v[4];
#pragma unroll
    for (int c = 0; c < 4; ++c) v[c] = row[c * 128];
    uint32_t sum = 0;
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const uint32_t q[4] = {v[c].x, v[c].y, v[c].z, v[c].w};
#pragma unroll
      for (int j = 0; j < 4; ++j)   // (|-128| is 128 as an unsigned byte)
        sum = __dp4a(__vabs4(q[j] ^ 0x80808080u), 0x01010101u, sum);
    }
    best = max(best, sum);
  }
  best = __reduce_max_sync(0xffffffffu, best);
  if ((threadIdx.x & 31) == 0 && best > 0) atomicMax(bound, static_cast<int32_t>(best));
}

// The row of x behind sorted row s, or -1.
__device__ __forceinline__ int64_t operand_row(const OperandJob& job, int64_t s) {
  int64_t row = s;
  if (job.order != nullptr) {
    const int slot = job.order[s];   // (written by the kernel before: no __ldg)
    if (slot < 0) return -1;
    row = job.k == 1 ? slot : slot / job.k;
  }
  return row < job.x_rows ? row : -1;
}
// Inputs 8c .. 8c + 7 of a row; those past K are zeros (their weights are too).
template <bool VEC>
__device__ __forceinline__ uint2 operand_load(const int8_t* src, int64_t c, int64_t K) {
  if constexpr (VEC)
    return c * 8 < K ? __ldg(reinterpret_cast<const uint2*>(src + c * 8)) : make_uint2(0, 0);
  uint32_t v[2] = {0, 0};
#pragma unroll
  for (int j = 0; j < 8; ++j)
    if (c * 8 + j < K)
      v[j / 4] |= static_cast<uint32_t>(static_cast<uint8_t>(__ldg(src + c * 8 + j)))
                  << (8 * (j % 4));
  return make_uint2(v[0], v[1]);
}
__device__ __forceinline__ uint4 operand_f16(uint2 w, __half2 minus) {
  w.x ^= 0x80808080u;
  w.y ^= 0x80808080u;
  return make_uint4(biased_to_f16x2(w.x, 0x4140, minus), biased_to_f16x2(w.x, 0x4342, minus),
                    biased_to_f16x2(w.y, 0x4140, minus), biased_to_f16x2(w.y, 0x4342, minus));
}

// The operand by whole warps: 32 x 8 inputs of a row a step, U steps at a time
// (their loads in flight together), the row looked up once for them; a step
// writes four whole 128-byte lines.  HBM's writes bound it: 8192 rows x 4096
// 12.8 us (67 MB written, 5.2 TB/s), 2048 rows 6.3 us.
template <int U, bool VEC>
__global__ void __launch_bounds__(256) tile_operand_kernel(const OperandJob job) {
  pdl_wait();
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
  const int64_t step = static_cast<int64_t>(gridDim.x) * blockDim.x;
  for (int64_t i = t; i < job.count_words; i += step) job.counts[i] = 0;
  // x - zp = (1024 + u) - (1152 + zp): integers below 2048, exact in f16
  const __half2 minus = __half2half2(__int2half_rn(1152 + job.zp));
  const uint32_t chunks = job.KB * 8;               // of 8 inputs
  const uint32_t segs = (chunks + U * 32 - 1) / (U * 32);
  const int64_t units = static_cast<int64_t>(job.R) * segs;
  int64_t s = (t >> 5) / segs;
  uint32_t seg = static_cast<uint32_t>((t >> 5) - s * segs);
  const int64_t rows_step = (step >> 5) / segs;
  const uint32_t seg_step = static_cast<uint32_t>((step >> 5) - rows_step * segs);
  for (int64_t u = t >> 5; u < units; u += step >> 5) {
    const int64_t row = operand_row(job, s);
    if (row >= 0) {
      const int8_t* src = job.x + row * job.K;
      uint2 w[U];
#pragma unroll
      for (int i = 0; i < U; ++i) {
        const uint32_t c = (seg * U + i) * 32 + lane;
        w[i] = c < chunks ? operand_load<VEC>(src, c, job.K) : make_uint2(0, 0);
      }
#pragma unroll
      for (int i = 0; i < U; ++i) {
        const uint32_t c = (seg * U + i) * 32 + lane;
        if (c < chunks)
          job.dst[(static_cast<int64_t>(c >> 3) * job.R + s) * 8 + (c & 7)] =
              operand_f16(w[i], minus);
      }
    }
    s += rows_step;
    seg += seg_step;
    if (seg >= segs) {
      seg -= segs;
      ++s;
    }
  }
}

// ---------------------------------------------------------------------------
// Adapters: h[s, j] = s_in * scaling[a] * sum_k (x[row(s), k] - zp) A[a][j, k]
// for the rows with an adapter, by m16n8k16 MMAs with ranks on M and rows on
// N.  The sum over k may take any order, so a thread's fragments of two MMAs
// are 8 consecutive inputs.  A CTA's warps, and the CTAs of a cluster while
// there are few, share K; their f32 sums are added in a fixed order, across
// the cluster through distributed shared memory.
//   lora_front_kernel, up to kMaxTileRows rows (one row tile): the rows come as
// they are, and 16 ranks of one adapter are a unit, taken where its first row
// is, for all of its rows, so that A is read once.  Loads go straight to
// registers, 4 steps of 32 inputs at once: what bounds it is latency (64 rows x
// 4096, 32 adapters of rank 16, 7.6 us).  The same launch writes the tile's
// operand and list.
//   lora_shrink_kernel, more rows: they come sorted by adapter, in the operand,
// and a unit is up to 32 rows of one adapter and all its ranks, 64 at a time.
// A's and the rows' k-blocks go through a ring in shared memory, their 16-byte
// chunks swizzled so that eight lanes' loads meet no bank twice (2048 rows x
// 4096, 8 adapters of rank 64, 20 us from cold memory, 31 when each 16 ranks
// were loaded straight to registers).
// ---------------------------------------------------------------------------
constexpr int kFrontThreads = 256;
constexpr int kFrontCluster = 8;   // CTAs that share one unit's K while units are few
constexpr int kFrontRows = 32;

template <bool F16>
__device__ __forceinline__ void mma_16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                          uint32_t b1) {
  if constexpr (F16)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

constexpr int kFrontWarps = kFrontThreads / 32;

struct ListShared {
  int32_t rows[kMaxTileRows];     // the rows this cluster takes, or a tile's rows' adapters
  int32_t held[kMaxTileRows];     // a tile's adapters
  int32_t warp_count[kFrontWarps];
};
struct FrontShared {
  float part[kFrontWarps][16][kFrontRows + 1];
  // the cluster's sums of this CTA's rows: [CTA][row][rank], written by each
  // (reading the others' took 10,000 cycles where writing to them takes 4,000)
  float sums[kFrontRows][16 + 1];
  ListShared list;
};

// Eight int8 inputs minus zp in the adapters' type (bf16 and f16 both hold
// integers up to 255 exactly).
template <bool F16>
__device__ __forceinline__ void widen_x8(uint2 w, int zp, uint32_t (&v)[4]) {
  if constexpr (F16) {
    const uint4 h = operand_f16(w, __half2half2(__int2half_rn(1152 + zp)));
    v[0] = h.x;
    v[1] = h.y;
    v[2] = h.z;
    v[3] = h.w;
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t h = j < 2 ? w.x >> (16 * j) : w.y >> (16 * (j - 2));
      v[j] = bf16x2_from_ints(static_cast<int8_t>(h & 0xff) - zp,
                              static_cast<int8_t>((h >> 8) & 0xff) - zp);
    }
  }
}

// This warp's share of K for 16 ranks and 8 * NT rows: the loads of U steps of
// 32 inputs go out together before any is used.
template <bool F16, int CL, bool VEC, int NT, int U>
__device__ __forceinline__ void front_products(const LoraJob& job, const uint16_t* A,
                                               const int64_t (&from)[4], int first,
                                               float (&acc)[4][4]) {
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int Kp = job.op.KB * 64;
  constexpr int kStep = CL * kFrontThreads;
  for (int k = first; k < Kp; k += U * kStep) {
    uint4 lo[U], hi[U];
    uint2 x[U][NT];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int k0 = k + u * kStep + t * 8;
      if (k + u * kStep < Kp) {
        lo[u] = __ldg(reinterpret_cast<const uint4*>(A + static_cast<int64_t>(g) * Kp + k0));
        hi[u] = __ldg(reinterpret_cast<const uint4*>(A + static_cast<int64_t>(g + 8) * Kp + k0));
#pragma unroll
        for (int n = 0; n < NT; ++n)
          x[u][n] = operand_load<VEC>(job.op.x + from[n] * job.op.K, k0 >> 3, job.op.K);
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (k + u * kStep < Kp) {
        const uint32_t a0[4] = {lo[u].x, hi[u].x, lo[u].y, hi[u].y};
        const uint32_t a1[4] = {lo[u].z, hi[u].z, lo[u].w, hi[u].w};
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          uint32_t v[4];
          widen_x8<F16>(x[u][n], job.op.zp, v);
          mma_16816<F16>(acc[n], a0, v[0], v[1]);
          mma_16816<F16>(acc[n], a1, v[2], v[3]);
        }
      }
  }
}

// h[s, j].  For dot products row by row: [R][ranks].  For MMAs: a block of
// [TN rows][16 leading terms, 16 trailing ones] for each adapter a tile t holds
// and 16 ranks, at (t + a) * rank16 + c (with the rows sorted by adapter,
// either t or a grows from one such pair to the next).  The MMAs read 10 bits of
// a term's fraction and cut off the rest, so both are rounded to that here: they
// miss h by its last place at most (not rounded, by three, and always towards
// zero).  From 2^127 on, where rounding could make an infinity, they are cut.
// Ranks from r on are zeros whatever the scaling is (0 times an infinite one
// would be NaN).
// s is row `local` of tile t.
__device__ __forceinline__ void store_h(const LoraJob& job, int s, int t, int local, int a, int j,
                                        float v) {
  if (j >= job.r) v = 0.0f;
  if (job.TN == 0) {
    job.h[static_cast<int64_t>(s) * job.rank16 * 16 + j] = v;
    return;
  }
  const int64_t block = static_cast<int64_t>(t + a) * job.rank16 + (j >> 4);
  float* at = job.h + (block * job.TN + local) * 32 + (j & 15);
  const uint32_t half = (__float_as_uint(v) & 0x7f000000u) == 0x7f000000u ? 0u : 0x1000u;
  const auto tf32 = [&](float f) {
    return __uint_as_float((__float_as_uint(f) + half) & 0xffffe000u);
  };
  const float hi = tf32(v);
  at[0] = hi;
  // (inf - inf would be NaN)
  at[16] = (__float_as_uint(hi) & 0x7f800000u) == 0x7f800000u ? 0.0f : tf32(__fsub_rn(v, hi));
}

// 16 ranks (block c) of adapter a for `count` <= 32 rows of the batch.  Every
// CTA of a cluster has arrived at its barrier once more than it has waited,
// here and on return: the others run, and their sums may be overwritten.
template <bool F16, int CL, bool VEC>
__device__ void front_rows(const LoraJob& job, FrontShared& sh, cg::cluster_group& cluster, int a,
                           int c, const int32_t* rows, int count) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int rank = CL > 1 ? cluster.block_rank() : 0;
  const uint16_t* A =
      job.a + (static_cast<int64_t>(a) * job.rank16 + c) * 16 * (job.op.KB * 64);
  float acc[4][4] = {};
  int64_t from[4];
#pragma unroll
  for (int n = 0; n < 4; ++n) {
    const int i = min(n * 8 + g, count - 1);   // rows past the last repeat it, unused
    from[n] = rows[i];
  }
  const int first = (rank * (kFrontThreads / 32) + warp) * 32;
  if (count <= 8) front_products<F16, CL, VEC, 1, 4>(job, A, from, first, acc);
  else front_products<F16, CL, VEC, 4, 2>(job, A, from, first, acc);
#pragma unroll
  for (int n = 0; n < 4; ++n)
#pragma unroll
    for (int j = 0; j < 4; ++j) sh.part[warp][g + (j >> 1) * 8][n * 8 + t * 2 + (j & 1)] = acc[n][j];
  __syncthreads();
  if constexpr (CL > 1) cluster_wait();
  constexpr int kRows = kFrontRows / CL;   // this CTA's share of the rows
  for (int i = threadIdx.x; i < 16 * kFrontRows; i += kFrontThreads) {
    const int j = i / kFrontRows, col = i % kFrontRows;
    float v = 0.0f;
#pragma unroll
    for (int w = 0; w < kFrontWarps; ++w) v += sh.part[w][j][col];
    float* to = &sh.sums[rank * kRows + col % kRows][j];
    if constexpr (CL > 1) to = cluster.map_shared_rank(to, col / kRows);
    if (col < count) *to = v;
  }
  if constexpr (CL > 1) cluster.sync(); else __syncthreads();
  for (int i0 = threadIdx.x; i0 < 16 * kRows; i0 += kFrontThreads) {
    const int j = i0 & 15, i = rank * kRows + (i0 >> 4);
    if (i < count) {
      float v = 0.0f;
#pragma unroll
      for (int q = 0; q < CL; ++q) v += sh.sums[q * kRows + (i0 >> 4)][j];
      store_h(job, rows[i], 0, rows[i], a, c * 16 + j, v * job.s_in * __ldg(job.scaling + a));
    }
  }
  if constexpr (CL > 1) cluster_arrive(); else __syncthreads();
}

__device__ __forceinline__ int adapter_of(const LoraJob& job, int s) {
  const int row = job.op.order != nullptr ? job.op.order[s] : s;
  const int a = __ldg(job.adapter_ids + row);
  return a >= 0 && a < job.L ? a : -1;
}

// Indices i < n whose flag is set, in order, into list; returns how many.
__device__ int block_compact(ListShared& sh, bool flag, int32_t value, int32_t* list) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t m = __ballot_sync(0xffffffffu, flag);
  if (lane == 0) sh.warp_count[warp] = __popc(m);
  __syncthreads();
  int before = 0, total = 0;
#pragma unroll
  for (int w = 0; w < kFrontThreads / 32; ++w) {
    if (w < warp) before += sh.warp_count[w];
    total += sh.warp_count[w];
  }
  if (flag) list[before + __popc(m & ((1u << lane) - 1u))] = value;
  __syncthreads();
  return total;
}

// A tile's adapters, each once, in the order of their first rows; and, where
// MMAs take them, zeros in the rows of h's blocks that are other adapters'.
// job.list_ctas CTAs share a tile's blocks.
__device__ void list_tile(const LoraJob& job, ListShared& sh, int cta) {
  const int tile = cta / job.list_ctas, part = cta % job.list_ctas;
  const int per = tile_rows(job.op.R, job.tiles), row0 = tile * per, n = min(per, job.op.R - row0);
  const int t = threadIdx.x;
  const int a = t < n ? adapter_of(job, row0 + t) : -1;
  if (t < n) sh.rows[t] = a;
  __syncthreads();
  bool first = a >= 0;
  if (job.op.order != nullptr) first = first && (t == 0 || sh.rows[t - 1] != a);
  else
    for (int i = 0; i < t && first; ++i) first = sh.rows[i] != a;
  __syncthreads();
  int32_t* list = job.lists + static_cast<int64_t>(tile) * job.list_stride;
  if (part == 0) {
    const int count = block_compact(sh, first, a, list + 1);
    if (t == 0) list[0] = count;
    if (job.ids_out != nullptr && t < n) job.ids_out[row0 + t] = a;
  }
  if (job.TN == 0) return;
  const int held = block_compact(sh, first, a, sh.held);
  const int blocks = held * job.rank16, rows = (n + 15) & ~15, lane = t & 31;
  // a warp a block, 4 rows of 128 bytes at a time
  for (int b = part * kFrontWarps + (t >> 5); b < blocks; b += job.list_ctas * kFrontWarps) {
    const int own = sh.held[b / job.rank16];
    float4* to = reinterpret_cast<float4*>(
        job.h + (static_cast<int64_t>(tile + own) * job.rank16 + b % job.rank16) * job.TN * 32);
    for (int i = lane >> 3; i < rows; i += 4)
      if (i >= n || sh.rows[i] != own) to[i * 8 + (lane & 7)] = make_float4(0.f, 0.f, 0.f, 0.f);
  }
}

// Blocks: job.shrink_ctas for h, then job.list_ctas for the list, the rest for
// the operand.
template <bool F16, int CL, bool VEC>
__global__ void __launch_bounds__(kFrontThreads, 2) lora_front_kernel(const LoraJob job) {
  __shared__ FrontShared sh;
  cg::cluster_group cluster = cg::this_cluster();
  pdl_wait();
  pdl_launch_dependents();
  const int R = job.op.R;
  int b = blockIdx.x;
  if (b < job.shrink_ctas) {
    // row w's adapter, if no earlier row has it
    const int u = b / CL, c = u % job.rank16, w = u / job.rank16;
    const int a = adapter_of(job, w);
    const int mine = static_cast<int>(threadIdx.x) < R ? adapter_of(job, threadIdx.x) : -1;
    const bool same = a >= 0 && mine == a;
    if (__syncthreads_or(same && static_cast<int>(threadIdx.x) < w) || a < 0) return;
    if constexpr (CL > 1) cluster_arrive();
    const int n = block_compact(sh.list, same, threadIdx.x, sh.list.rows);
    for (int i = 0; i < n; i += kFrontRows)
      front_rows<F16, CL, VEC>(job, sh, cluster, a, c, sh.list.rows + i, min(kFrontRows, n - i));
    if constexpr (CL > 1) cluster_wait();
    return;
  }
  b -= job.shrink_ctas;
  if (b < job.list_ctas) {
    list_tile(job, sh.list, b);
    return;
  }
  b -= job.list_ctas;
  const uint32_t t = b * kFrontThreads + threadIdx.x;   // (some thousand CTAs at most)
  const uint32_t step = (gridDim.x - job.shrink_ctas - job.list_ctas) * kFrontThreads;
  for (int64_t i = t; i < job.op.count_words; i += step) job.op.counts[i] = 0;
  const __half2 minus = __half2half2(__int2half_rn(1152 + job.op.zp));
  const uint32_t chunks = job.op.KB * 8;
  for (RowItems at(t, step, chunks); at.row < R; at.next()) {
    const uint32_t c = at.item;
    job.op.dst[(static_cast<int64_t>(c >> 3) * R + at.row) * 8 + (c & 7)] =
        operand_f16(operand_load<VEC>(job.op.x + at.row * job.op.K, c, job.op.K), minus);
  }
}

// 16 ranks of 4 blocks, and 32 rows, of one k-block
constexpr int kShrinkBlocks = 4, kShrinkStages = 4;
constexpr int kShrinkStage = (kShrinkBlocks * 16 + kFrontRows) * 128;

struct ShrinkShared {
  float part[kFrontWarps][16][kFrontRows + 1];
  float sums[kFrontRows][kShrinkBlocks * 16 + 1];   // as in FrontShared
  ListShared list;
  int32_t piece[3];                            // adapter, first row, rows
};

// Where a row's 16-byte chunk of a 128-byte k-block lies: rows 2i and 2i + 1
// keep their chunks 0 to 3 in different halves.
__device__ __forceinline__ uint32_t shrink_at(int row, int chunk) {
  return row * 128 + ((chunk ^ ((row & 1) << 2 | ((row >> 1) & 3))) << 4);
}

__device__ __forceinline__ uint32_t f16x2_to_bf16x2(uint32_t v) {
  const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&v));
  const __nv_bfloat162 b = __floats2bfloat162_rn(f.x, f.y);   // integers up to 255: exact
  return *reinterpret_cast<const uint32_t*>(&b);
}

// Unit u's piece of 32 rows at most: adapters in turn, each cut into pieces.
__device__ bool find_piece(const LoraJob& job, ShrinkShared& sh, int u) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int before = 0;
  for (int a0 = 0; a0 < job.L; a0 += kFrontThreads) {
    const int a = a0 + threadIdx.x;
    int first = 0, rows = 0;
    if (a < job.L) {
      first = job.offsets[a];
      rows = job.offsets[a + 1] - first;
    }
    const int n = (rows + kFrontRows - 1) / kFrontRows;
    int incl = n;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, incl, d);
      if (lane >= d) incl += v;
    }
    if (lane == 31) sh.list.warp_count[warp] = incl;
    __syncthreads();
    int all = 0;
#pragma unroll
    for (int w = 0; w < kFrontWarps; ++w) {
      if (w < warp) incl += sh.list.warp_count[w];
      all += sh.list.warp_count[w];
    }
    const int i = u - (before + incl - n);
    if (i >= 0 && i < n) {
      sh.piece[0] = a;
      sh.piece[1] = first + i * kFrontRows;
      sh.piece[2] = min(kFrontRows, rows - i * kFrontRows);
    }
    __syncthreads();
    before += all;
    if (u < before) return true;
  }
  return false;
}

// Blocks: job.shrink_ctas for h, in clusters, then job.list_ctas per row tile
// for its list.
template <bool F16>
__global__ void __launch_bounds__(kFrontThreads, 2)
    lora_shrink_kernel(const __grid_constant__ LoraJob job) {
  extern __shared__ __align__(128) uint8_t ring[];
  __shared__ ShrinkShared sh;
  pdl_wait();
  pdl_launch_dependents();
  if (static_cast<int>(blockIdx.x) >= job.shrink_ctas) {
    if (static_cast<int>(blockIdx.x) - job.shrink_ctas < job.tiles * job.list_ctas)
      list_tile(job, sh.list, blockIdx.x - job.shrink_ctas);
    return;
  }
  cg::cluster_group cluster = cg::this_cluster();
  const int CL = cluster.num_blocks(), rank = cluster.block_rank();
  if (!find_piece(job, sh, blockIdx.x / CL)) return;   // (all of a cluster or none)
  cluster_arrive();
  const int a = sh.piece[0], row0 = sh.piece[1], count = sh.piece[2];
  const float scale = job.s_in * __ldg(job.scaling + a);
  const int per = tile_rows(job.op.R, job.tiles), tile0 = row0 / per;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int rows = kFrontRows / CL;
  const int KB = job.op.KB, kb0 = rank * KB / CL, steps = (rank + 1) * KB / CL - kb0;
  const int64_t Kp = static_cast<int64_t>(KB) * 64;
  const uint32_t ring0 = smem_u32(ring);
  for (int c0 = 0; c0 < job.rank16; c0 += kShrinkBlocks) {
    // a block of 16 ranks to each warp, the warps of one sharing K
    const int blocks = min(kShrinkBlocks, job.rank16 - c0);
    const int spread = blocks == 3 ? 4 : blocks, mine = warp % spread, k_of = warp / spread;
    const int shares = kFrontWarps / spread;
    const uint16_t* A = job.a + (static_cast<int64_t>(a) * job.rank16 + c0) * 16 * Kp;
    const auto fill = [&](int i) {
      if (i < steps) {
        const uint32_t st = ring0 + (i % kShrinkStages) * kShrinkStage;
        const int row = threadIdx.x >> 3, chunk = threadIdx.x & 7;
        const uint4* x = job.op.dst +
                         (static_cast<int64_t>(kb0 + i) * job.op.R + row0 + min(row, count - 1)) * 8;
        cp_async16(st + shrink_at(row, chunk), x + chunk);
#pragma unroll
        for (int j = 0; j < kShrinkBlocks / 2; ++j) {
          const int r = row + j * 32;
          if (r < blocks * 16)
            cp_async16(st + shrink_at(kFrontRows + r, chunk),
                       A + r * Kp + (kb0 + i) * 64 + chunk * 8);
        }
      }
      cp_async_commit();
    };
    float acc[4][4] = {};
    for (int i = 0; i < kShrinkStages - 1; ++i) fill(i);
    for (int i = 0; i < steps; ++i) {
      cp_async_wait<kShrinkStages - 2>();
      __syncthreads();
      fill(i + kShrinkStages - 1);
      const uint32_t st = ring0 + (i % kShrinkStages) * kShrinkStage;
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        if (mine >= blocks || (i * 2 + half) % shares != k_of) continue;
        const int chunk = half * 4 + t;
        const uint4 lo = lds128(st + shrink_at(kFrontRows + mine * 16 + g, chunk));
        const uint4 hi = lds128(st + shrink_at(kFrontRows + mine * 16 + g + 8, chunk));
        const uint32_t a0[4] = {lo.x, hi.x, lo.y, hi.y}, a1[4] = {lo.z, hi.z, lo.w, hi.w};
#pragma unroll
        for (int n = 0; n < 4; ++n) {
          uint4 x = lds128(st + shrink_at(n * 8 + g, chunk));
          if constexpr (!F16) {
            x.x = f16x2_to_bf16x2(x.x);
            x.y = f16x2_to_bf16x2(x.y);
            x.z = f16x2_to_bf16x2(x.z);
            x.w = f16x2_to_bf16x2(x.w);
          }
          mma_16816<F16>(acc[n], a0, x.x, x.y);
          mma_16816<F16>(acc[n], a1, x.z, x.w);
        }
      }
    }
    cp_async_wait<0>();
#pragma unroll
    for (int n = 0; n < 4; ++n)
#pragma unroll
      for (int j = 0; j < 4; ++j)
        sh.part[warp][g + (j >> 1) * 8][n * 8 + t * 2 + (j & 1)] = acc[n][j];
    __syncthreads();
    cluster_wait();   // the others run, and have read the sums of the ranks before
    for (int i = threadIdx.x; i < blocks * 16 * kFrontRows; i += kFrontThreads) {
      const int j = i / kFrontRows, col = i % kFrontRows;
      float v = 0.0f;
      for (int k = 0; k < shares; ++k) v += sh.part[k * spread + j / 16][j % 16][col];
      if (col < count)
        *cluster.map_shared_rank(&sh.sums[rank * rows + col % rows][j], col / rows) = v;
    }
    cluster.sync();
    // this CTA's share of the rows, a rank a thread (code that runs once: few
    // instructions, for they cost more to fetch than to execute)
    const int j = threadIdx.x % (kShrinkBlocks * 16);
    const int i1 = min(count, (rank + 1) * rows);
    if (j < blocks * 16)
      for (int i = rank * rows + threadIdx.x / (kShrinkBlocks * 16); i < i1;
           i += kFrontThreads / (kShrinkBlocks * 16)) {
        float v = 0.0f;
        for (int q = 0; q < CL; ++q) v += sh.sums[q * rows + i % rows][j];
        int t = tile0, local = row0 - tile0 * per + i;
        while (local >= per) {
          local -= per;
          ++t;
        }
        store_h(job, row0 + i, t, local, a, c0 * 16 + j, v * scale);
      }
    cluster_arrive();
  }
  cluster_wait();
}

// Adapter matrices, padded with zeros: A -> [L][16 rank16][64 KB], and
// B -> [L][NB][rank16][2][128][8] (8-rank chunks of all 128 channels).  A tile
// multiplies every adapter it holds by all of its rows, zeros standing for the
// rows of others, so an infinity or NaN of B must not enter the product:
// those entries become zeros, and the adapter's scaling NaN
// (lora_scaling_kernel), which makes its own rows NaN and no others.
__device__ __forceinline__ bool finite16(uint16_t v, uint32_t exponent) {
  return (v & exponent) != exponent;
}

__global__ void __launch_bounds__(256) lora_scaling_kernel(const uint16_t* __restrict__ B,
                                                           const float* __restrict__ scaling,
                                                           int64_t per, uint32_t exponent,
                                                           float* __restrict__ s_out) {
  pdl_wait();
  bool bad = false;
  for (int64_t i = threadIdx.x; i < per; i += blockDim.x)
    bad |= !finite16(B[blockIdx.x * per + i], exponent);
  bad = __syncthreads_or(bad);
  if (threadIdx.x == 0)
    s_out[blockIdx.x] = bad ? __int_as_float(0x7fffffff) : scaling[blockIdx.x];
}

__global__ void __launch_bounds__(256) pack_lora_kernel(const uint16_t* __restrict__ A,
                                                        const uint16_t* __restrict__ B,
                                                        uint32_t exponent, int64_t L, int64_t r,
                                                        int64_t N, int64_t K, int64_t rank16,
                                                        int64_t NB, int64_t Kp,
                                                        uint16_t* __restrict__ a_out,
                                                        uint16_t* __restrict__ b_out) {
  pdl_wait();
  const int64_t t = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
  const int64_t step = static_cast<int64_t>(gridDim.x) * blockDim.x;
  const int64_t rp = rank16 * 16;
  for (int64_t i = t; i < L * rp * Kp; i += step) {
    const int64_t k = i % Kp, j = i / Kp % rp, l = i / Kp / rp;
    a_out[i] = (k < K && j < r) ? A[(l * r + j) * K + k] : 0;
  }
  for (int64_t i = t; i < L * NB * rank16 * 2048; i += step) {
    const int64_t w = i & 7, row = (i >> 3) & 127, half = (i >> 10) & 1;
    int64_t q = i >> 11;
    const int64_t c = q % rank16;
    q /= rank16;
    const int64_t n = (q % NB) * 128 + row, l = q / NB, j = c * 16 + half * 8 + w;
    const uint16_t v = (n < N && j < r) ? B[(l * N + n) * r + j] : 0;
    b_out[i] = finite16(v, exponent) ? v : 0;
  }
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

cudaError_t launch_tile_weight_bound(const uint8_t* packed, int64_t tiles, int32_t* bound,
                                     cudaStream_t s) {
  const cudaError_t e = cudaMemsetAsync(bound, 0, sizeof(int32_t), s);
  if (e != cudaSuccess) return e;
  return launch_pdl(tile_weight_bound_kernel, blocks_for(tiles * 128), 256, 0, s,
                    reinterpret_cast<const uint4*>(packed), tiles, bound);
}

cudaError_t launch_tile_operand(const OperandJob& job, cudaStream_t s) {
  const auto go = [&](auto u, auto vec) {
    constexpr int U = decltype(u)::value;
    const int64_t units = static_cast<int64_t>(job.R) * ((job.KB * 8 + U * 32 - 1) / (U * 32));
    return launch_pdl(tile_operand_kernel<U, decltype(vec)::value>,
                      blocks_for(std::max<int64_t>(units * 32, job.count_words)), 256, 0, s, job);
  };
  const auto with = [&](auto vec) {
    // one step a warp while that still leaves SMs idle
    return static_cast<int64_t>(job.R) * job.KB < 64 * device_sm_count()
               ? go(std::integral_constant<int, 1>(), vec)
               : go(std::integral_constant<int, 4>(), vec);
  };
  return rows_vec8(job) ? with(std::true_type()) : with(std::false_type());
}

cudaError_t launch_pack_lora(const void* A, const void* B, const float* scaling, bool f16,
                             int64_t L, int64_t r, int64_t N, int64_t K, void* a_out, void* b_out,
                             float* s_out, cudaStream_t s) {
  const int64_t rank16 = (r + 15) / 16, NB = (N + 127) / 128, Kp = round_up(K, 64);
  const uint32_t exponent = f16 ? 0x7c00u : 0x7f80u;
  const auto* b = static_cast<const uint16_t*>(B);
  cudaError_t e = launch_pdl(lora_scaling_kernel, static_cast<int>(L), 256, 0, s, b, scaling, N * r,
                             exponent, s_out);
  if (e != cudaSuccess) return e;
  return launch_pdl(pack_lora_kernel, blocks_for(L * rank16 * 16 * Kp), 256, 0, s,
                    static_cast<const uint16_t*>(A), b, exponent, L, r, N, K, rank16, NB, Kp,
                    static_cast<uint16_t*>(a_out), static_cast<uint16_t*>(b_out));
}

namespace {

// Rows sorted by adapter: the operand, then h from it.
template <bool F16>
cudaError_t launch_sorted(LoraJob job, cudaStream_t s) {
  cudaError_t e = launch_tile_operand(job.op, s);
  if (e != cudaSuccess) return e;
  static DeviceOnce once;
  e = once.run([] {
    return cudaFuncSetAttribute(lora_shrink_kernel<F16>,
                                cudaFuncAttributeMaxDynamicSharedMemorySize,
                                kShrinkStages * kShrinkStage);
  });
  if (e != cudaSuccess) return e;
  const int units = job.op.R / kFrontRows + std::min(job.L, job.op.R);
  // K is cut over a cluster while all CTAs are resident at once, two an SM
  // (the lists' behind those for h cost their whole time again), and a tile's
  // list is shared by those that are left
  const int slots = 2 * device_sm_count();
  int cl = kFrontCluster;
  while (cl > 1 && units * cl + job.tiles > slots) cl /= 2;
  job.shrink_ctas = units * cl;
  job.list_ctas = std::max(1, std::min(4, (slots - job.shrink_ctas) / job.tiles));
  return launch_pdl_cluster(lora_shrink_kernel<F16>,
                            static_cast<int>(round_up(job.shrink_ctas + job.tiles * job.list_ctas, cl)),
                            kFrontThreads, kShrinkStages * kShrinkStage, cl, s, job);
}

}  // namespace

cudaError_t launch_lora_front(LoraJob job, bool f16, cudaStream_t s) {
  if (job.op.order != nullptr)
    return f16 ? launch_sorted<true>(job, s) : launch_sorted<false>(job, s);
  // K is cut over 8 CTAs while the units alone would leave SMs without one
  const int cl = job.op.R * job.rank16 <= device_sm_count() ? kFrontCluster : 1;
  job.shrink_ctas = job.op.R * job.rank16 * cl;
  job.list_ctas = 4;
  const int copy = blocks_for(
      std::max<int64_t>(static_cast<int64_t>(job.op.R) * job.op.KB * 8, job.op.count_words));
  const int grid = static_cast<int>(round_up(job.shrink_ctas + job.list_ctas + copy, cl));
  const auto go = [&](auto half, auto vec) {
    constexpr bool F16 = decltype(half)::value, VEC = decltype(vec)::value;
    return cl == 1 ? launch_pdl(lora_front_kernel<F16, 1, VEC>, grid, kFrontThreads, 0, s, job)
                   : launch_pdl_cluster(lora_front_kernel<F16, kFrontCluster, VEC>, grid,
                                        kFrontThreads, 0, kFrontCluster, s, job);
  };
  const auto with = [&](auto half) {
    return rows_vec8(job.op) ? go(half, std::true_type()) : go(half, std::false_type());
  };
  return f16 ? with(std::true_type()) : with(std::false_type());
}

}  // namespace q8
