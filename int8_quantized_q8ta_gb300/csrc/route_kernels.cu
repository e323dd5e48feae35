// route_kernels.cu -- tokens sorted by expert and back, with weights applied,
// and the gradients (sm_103a).
//
// T tokens choose k experts each; slot f = t*k + j holds the id e_f.  A slot
// whose id lies outside [0, E) is dropped.
//   sort     stable by id: offsets[e] = #{f : 0 <= e_f < e}; position[f] is
//            slot f's row, order[row] its inverse; -1 marks a dropped slot in
//            position and the rows from offsets[E] on in order
//   gather   xs[row] = x[order[row] / k], zeros from row offsets[E] on
//   spread   the sum that brings rows back to tokens, with weights (combine)
//            or without (the gather's gradient):
//            y[t] = sum_j w[t,j] * z[position[t,j]] over the kept slots
//   combine's gradient  dz[row] = w[order[row]] * dy[order[row] / k] and
//            dw[t,j] = <dy[t], z[position[t,j]]>
// Sums are f32, taken in slot order j = 0, 1, ..., rounded once to the row
// type.  No atomics on global memory: results do not depend on timing.
//   All but the sort are bound by HBM in long batches and by the latency of
// position -> row -> row in short ones.  Measured (calls one after another in a
// graph, three sets of inputs in turn; 6.8 TB/s is a plain copy): rows of 4096
// bf16, 2048 tokens of 4 experts: gather 14.3 us (84 MB, 5.9 TB/s), its gradient
// 16.3 (5.2); 4096 tokens of 8: gather 49.0 us (302 MB, 6.2 TB/s), combine 49.0
// (6.2), its gradient 88.5 (570 MB, 6.4).  Rows that are no multiple of 16 bytes
// are combined element by element: 3885 rows of 1001 halfs, combine 4.4 and its
// gradient 7.2 us (2.1 and 2.4 TB/s), of 1008 halfs 2.95 and 4.2.
#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>
#include <initializer_list>
#include <type_traits>

#include "device_common.cuh"
#include "q8ta_internal.h"
#include "rows_internal.h"

namespace q8 {

namespace cg = cooperative_groups;

namespace {

// ---------------------------------------------------------------------------
// sort: a counting sort by one cluster.  Each CTA owns a contiguous run of
// slots and each of its warps a contiguous part of that run, so a slot's row
// is (all slots of lower experts) + (its expert's slots in earlier CTAs) +
// (in earlier warps of its CTA) + (earlier in its warp): stable by
// construction.  The CTAs exchange their E + 1 totals through distributed
// shared memory; nothing but the ids is read from global memory.  A warp's
// slots of one expert are found by one ballot for each bit of the id (a match
// instruction takes as long as there are different ids).  Latency bounds it (in a
// graph, as above): 8 slots 3.0 us, 1024 4.8, 8192 5.1, 32768 6.6, and from there
// on the work of 8 CTAs, the most a portable cluster has: 262144 slots 26 us.
// ---------------------------------------------------------------------------
constexpr int kSortMaxWarps = 32;
constexpr int kSortKeys = 4;              // ids a thread has in flight

// The groups of slots f, f + 32, ...: experts, E for dropped, -1 from hi on.
__device__ __forceinline__ void sort_keys(const int32_t* ids, int64_t f, int64_t hi, int E,
                                          int (&key)[kSortKeys]) {
#pragma unroll
  for (int i = 0; i < kSortKeys; ++i) key[i] = f + i * 32 < hi ? __ldg(ids + f + i * 32) : -2;
#pragma unroll
  for (int i = 0; i < kSortKeys; ++i)
    key[i] = f + i * 32 >= hi ? -1 : key[i] >= 0 && key[i] < E ? key[i] : E;
}

// The sort by this cluster.  write: into global memory; rows, if not null, gets
// each slot's position too.  Returns the kept slots.
__device__ __forceinline__ int sort_slots(const int32_t* __restrict__ ids, int64_t R, int E,
                                          int32_t* __restrict__ order,
                                          int32_t* __restrict__ position,
                                          int32_t* __restrict__ offsets, bool keep_dropped,
                                          bool write, int32_t* sm, int32_t* rows) {
  const int G = E + 1;                        // groups: the experts and the dropped slots
  const int warps = blockDim.x >> 5, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int32_t* hist = sm;                         // [warps][G]
  int32_t* total = sm + warps * G;            // [G], read by the other CTAs
  int32_t* start = total + G;                 // [G]
  __shared__ int32_t carry[kSortMaxWarps];
  cg::cluster_group cluster = cg::this_cluster();
  const int ctas = cluster.num_blocks(), rank = cluster.block_rank();

  for (int i = threadIdx.x; i < warps * G; i += blockDim.x) hist[i] = 0;
  // slots per warp, a multiple of 32 so that only the last run is ragged
  const int64_t per = ((R + static_cast<int64_t>(ctas) * warps * 32 - 1) /
                       (static_cast<int64_t>(ctas) * warps * 32)) * 32;
  const int64_t lo = (static_cast<int64_t>(rank) * warps + warp) * per;
  const int64_t hi = min(R, lo + per);
  __syncthreads();
  pdl_wait();
  pdl_launch_dependents();
  int32_t* mine = hist + warp * G;
  for (int64_t f0 = lo; f0 < hi; f0 += 32 * kSortKeys) {
    int key[kSortKeys];
    sort_keys(ids, f0 + lane, hi, E, key);
#pragma unroll
    for (int i = 0; i < kSortKeys; ++i)
      if (key[i] >= 0) atomicAdd(&mine[key[i]], 1);
  }
  __syncthreads();
  for (int g = threadIdx.x; g < G; g += blockDim.x) {
    int32_t sum = 0;
    for (int w0 = 0; w0 < warps; w0 += 8) {
      int32_t c[8];
#pragma unroll
      for (int w = 0; w < 8; ++w) c[w] = hist[(w0 + w) * G + g];
#pragma unroll
      for (int w = 0; w < 8; ++w) {
        hist[(w0 + w) * G + g] = sum;
        sum += c[w];
      }
    }
    total[g] = sum;
  }
  cluster.sync();
  // exclusive scan over the groups of the cluster's totals, a block of
  // threads at a time
  int32_t before_all = 0;
  for (int g0 = 0; g0 < G; g0 += blockDim.x) {
    const int g = g0 + threadIdx.x;
    int32_t all = 0, earlier = 0;
    if (g < G)
#pragma unroll
      for (int c = 0; c < 8; ++c) {
        const int32_t v = c < ctas ? *cluster.map_shared_rank(total + g, c) : 0;
        if (c < rank) earlier += v;
        all += v;
      }
    int32_t incl = all;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int32_t v = __shfl_up_sync(0xffffffffu, incl, d);
      if (lane >= d) incl += v;
    }
    if (lane == 31) carry[warp] = incl;
    __syncthreads();
    const int32_t sum = lane < warps ? carry[lane] : 0;
    const int32_t add = before_all + __reduce_add_sync(0xffffffffu, lane < warp ? sum : 0);
    before_all += __reduce_add_sync(0xffffffffu, sum);
    const int32_t excl = add + incl - all;
    if (g < G) {
      start[g] = excl + earlier;
      if (rank == 0 && write) offsets[g] = excl;   // offsets[E]: the kept slots
    }
    __syncthreads();
  }
  cluster.sync();                             // totals stay readable until every CTA is done
  for (int64_t f0 = lo; f0 < hi; f0 += 32 * kSortKeys) {
    int key[kSortKeys];
    uint32_t peers[kSortKeys];                // the warp's lanes with the same key
    sort_keys(ids, f0 + lane, hi, E, key);
#pragma unroll
    for (int i = 0; i < kSortKeys; ++i) peers[i] = __ballot_sync(0xffffffffu, key[i] >= 0);
    for (int bit = 1; bit <= E; bit <<= 1) {
#pragma unroll
      for (int i = 0; i < kSortKeys; ++i) {
        const uint32_t set = __ballot_sync(0xffffffffu, key[i] & bit);
        peers[i] &= key[i] & bit ? set : ~set;
      }
    }
#pragma unroll
    for (int i = 0; i < kSortKeys; ++i) {
      const int rank_in = __popc(peers[i] & ((1u << lane) - 1u));
      int32_t row = 0;
      if (key[i] >= 0) row = start[key[i]] + mine[key[i]] + rank_in;
      __syncwarp();
      if (key[i] >= 0 && rank_in == 0) mine[key[i]] += __popc(peers[i]);
      __syncwarp();
      if (key[i] >= 0) {
        const int64_t f = f0 + i * 32 + lane;
        const int32_t at = key[i] < E ? row : -1;
        if (write) {
          order[row] = key[i] < E || keep_dropped ? static_cast<int32_t>(f) : -1;
          position[f] = at;
        }
        if (rows != nullptr) rows[f] = at;
      }
    }
  }
  return start[E];
}

__global__ void __launch_bounds__(1024) expert_sort_kernel(const int32_t* __restrict__ ids,
                                                           int64_t R, int E,
                                                           int32_t* __restrict__ order,
                                                           int32_t* __restrict__ position,
                                                           int32_t* __restrict__ offsets,
                                                           bool keep_dropped) {
  extern __shared__ int32_t sm[];
  sort_slots(ids, R, E, order, position, offsets, keep_dropped, true, sm, nullptr);
}

// ---------------------------------------------------------------------------
// rows as vectors: VB bytes of T at a time
// ---------------------------------------------------------------------------
template <int VB> struct VecOf;
template <> struct VecOf<16> { using type = uint4; };
template <> struct VecOf<8> { using type = uint2; };
template <> struct VecOf<4> { using type = uint32_t; };
template <> struct VecOf<2> { using type = uint16_t; };
template <> struct VecOf<1> { using type = uint8_t; };

template <typename T> __device__ __forceinline__ float to_f32(T v);
template <> __device__ __forceinline__ float to_f32<float>(float v) { return v; }
template <> __device__ __forceinline__ float to_f32<__half>(__half v) { return __half2float(v); }
template <> __device__ __forceinline__ float to_f32<__nv_bfloat16>(__nv_bfloat16 v) {
  return __bfloat162float(v);
}
template <typename T> __device__ __forceinline__ T from_f32(float v);
template <> __device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <> __device__ __forceinline__ __half from_f32<__half>(float v) {
  return __float2half_rn(v);
}
template <> __device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) {
  return __float2bfloat16_rn(v);
}

template <typename T, int VB>
union Pack {
  typename VecOf<VB>::type v;
  T e[VB / sizeof(T)];
  __device__ Pack() {}
};

// Zeros in the rows from `kept` on (dropped slots), by whole warps.
template <int VB>
__device__ __forceinline__ void zero_tail(typename VecOf<VB>::type* rows, int64_t V, int64_t R,
                                          int kept, int64_t warp_id, int64_t num_warps, int lane) {
  typename VecOf<VB>::type zero{};
  for (int64_t s = max(0, kept) + warp_id; s < R; s += num_warps)
    for (int64_t c = lane; c < V; c += 32) rows[s * V + c] = zero;
}

// gather: a warp takes U*32 vectors of one token's row, read once and written
// to each of the token's kept rows (k writes to one read: slots in sorted order
// would read every row k times).
template <int VB, int U>
__device__ __forceinline__ void gather_rows(const typename VecOf<VB>::type* __restrict__ x,
                                            int64_t T, int k, int64_t V, const int32_t* position,
                                            int kept, typename VecOf<VB>::type* __restrict__ xs) {
  const int lane = threadIdx.x & 31;
  const int64_t warp_id = (static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x) >> 5;
  const int64_t num_warps = (static_cast<int64_t>(gridDim.x) * blockDim.x) >> 5;
  const int64_t segs = (V + U * 32 - 1) / (U * 32);
  for (int64_t u = warp_id; u < T * segs; u += num_warps) {
    const int64_t t = u / segs, c0 = (u - t * segs) * (U * 32) + lane;
    typename VecOf<VB>::type v[U];
#pragma unroll
    for (int i = 0; i < U; ++i)
      if (c0 + i * 32 < V) v[i] = __ldg(x + t * V + c0 + i * 32);
    for (int j = 0; j < k; ++j) {
      const int64_t s = position[t * k + j];
      if (s < 0 || s >= T * k) continue;
#pragma unroll
      for (int i = 0; i < U; ++i)
        if (c0 + i * 32 < V) xs[s * V + c0 + i * 32] = v[i];
    }
  }
  zero_tail<VB>(xs, V, T * k, kept, warp_id, num_warps, lane);
}

template <int VB, int U>
__global__ void __launch_bounds__(256) expert_gather_kernel(
    const typename VecOf<VB>::type* __restrict__ x, int64_t T, int k, int64_t V,
    const int32_t* __restrict__ position, const int32_t* __restrict__ offsets, int E,
    typename VecOf<VB>::type* __restrict__ xs) {
  pdl_wait();
  pdl_launch_dependents();
  gather_rows<VB, U>(x, T, k, V, position, __ldg(offsets + E), xs);
}

// Both for few slots: every CTA sorts them all for itself and moves its share
// of the rows, one launch instead of two in a row (8 slots of 4096 bytes 3.9
// instead of 4.7 us).
constexpr int kDispatchSlots = 256;

template <int VB, int U>
__global__ void __launch_bounds__(256) expert_dispatch_kernel(
    const typename VecOf<VB>::type* __restrict__ x, const int32_t* __restrict__ ids, int64_t T,
    int k, int64_t V, int E, int32_t* __restrict__ order, int32_t* __restrict__ position,
    int32_t* __restrict__ offsets, typename VecOf<VB>::type* __restrict__ xs) {
  extern __shared__ int32_t sm[];
  __shared__ int32_t rows[kDispatchSlots];
  const int kept = sort_slots(ids, T * k, E, order, position, offsets, false, blockIdx.x == 0, sm,
                              rows);
  __syncthreads();
  gather_rows<VB, U>(x, T, k, V, rows, kept, xs);
}

// spread: a warp takes U*32 vectors of one token's sum, S slots' loads in
// flight (one slot after another took 15 instead of 10.7 us for 777 tokens'
// combine and its gradient, 37 instead of 35 for 2048 tokens' dispatch and
// its).  w: null for ones.
template <typename T, int VB, int U, int S>
__global__ void __launch_bounds__(256) expert_spread_kernel(
    const typename VecOf<VB>::type* __restrict__ z, const float* __restrict__ w, int64_t Tn, int k,
    int64_t V, const int32_t* __restrict__ position, typename VecOf<VB>::type* __restrict__ y) {
  constexpr int N = VB / sizeof(T);
  pdl_wait();
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31;
  const int64_t warp_id = (static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x) >> 5;
  const int64_t num_warps = (static_cast<int64_t>(gridDim.x) * blockDim.x) >> 5;
  const int64_t segs = (V + U * 32 - 1) / (U * 32);
  for (int64_t u = warp_id; u < Tn * segs; u += num_warps) {
    const int64_t t = u / segs, c0 = (u - t * segs) * (U * 32) + lane;
    float acc[U][N];
#pragma unroll
    for (int i = 0; i < U; ++i)
#pragma unroll
      for (int n = 0; n < N; ++n) acc[i][n] = 0.0f;
    for (int j0 = 0; j0 < k; j0 += 32) {
      // 32 slots' rows and weights, a lane each
      int32_t row = -1;
      float weight = 1.0f;
      if (j0 + lane < k) {
        row = __ldg(position + t * k + j0 + lane);
        if (w != nullptr) weight = __ldg(w + t * k + j0 + lane);
      }
      if (row >= Tn * k) row = -1;
      for (int j = 0; j < min(32, k - j0); j += S) {
        int32_t from[S];
        Pack<T, VB> p[S][U];
#pragma unroll
        for (int q = 0; q < S; ++q) {
          from[q] = __shfl_sync(0xffffffffu, row, j + q);   // -1 past the last slot
          if (from[q] >= 0)
#pragma unroll
            for (int i = 0; i < U; ++i)
              if (c0 + i * 32 < V) p[q][i].v = __ldg(z + from[q] * V + c0 + i * 32);
        }
#pragma unroll
        for (int q = 0; q < S; ++q) {
          const float wj = __shfl_sync(0xffffffffu, weight, j + q);
          if (from[q] >= 0)
#pragma unroll
            for (int i = 0; i < U; ++i)
              if (c0 + i * 32 < V)
#pragma unroll
                for (int n = 0; n < N; ++n)
                  acc[i][n] = fmaf(wj, to_f32<T>(p[q][i].e[n]), acc[i][n]);
        }
      }
    }
#pragma unroll
    for (int i = 0; i < U; ++i)
      if (c0 + i * 32 < V) {
        Pack<T, VB> p;
#pragma unroll
        for (int n = 0; n < N; ++n) p.e[n] = from_f32<T>(acc[i][n]);
        y[t * V + c0 + i * 32] = p.v;
      }
  }
}

// combine's gradient: a warp takes one slot, its whole row, U vectors at a time:
// dz is the token's dy times the slot's weight, dw the dot of dy with the
// slot's z.  dy comes from L2 for all but a token's first slot.
template <typename T, int VB, int U>
__global__ void __launch_bounds__(256) expert_combine_bwd_kernel(
    const typename VecOf<VB>::type* __restrict__ dy, const typename VecOf<VB>::type* __restrict__ z,
    const float* __restrict__ w, int64_t R, int k, int64_t V, const int32_t* __restrict__ position,
    const int32_t* __restrict__ offsets, int E, typename VecOf<VB>::type* __restrict__ dz,
    float* __restrict__ dw) {
  constexpr int N = VB / sizeof(T);
  pdl_wait();
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31;
  const int64_t warp_id = (static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x) >> 5;
  const int64_t num_warps = (static_cast<int64_t>(gridDim.x) * blockDim.x) >> 5;
  for (int64_t f = warp_id; f < R; f += num_warps) {
    const int64_t s = __ldg(position + f), t = f / k;
    float dot = 0.0f;
    if (s >= 0 && s < R) {
      const float wf = __ldg(w + f);
      for (int64_t c0 = lane; c0 < V; c0 += U * 32) {
        Pack<T, VB> a[U], b[U];
#pragma unroll
        for (int i = 0; i < U; ++i)
          if (c0 + i * 32 < V) {
            a[i].v = __ldg(dy + t * V + c0 + i * 32);
            b[i].v = __ldg(z + s * V + c0 + i * 32);
          }
#pragma unroll
        for (int i = 0; i < U; ++i)
          if (c0 + i * 32 < V) {
            Pack<T, VB> o;
#pragma unroll
            for (int n = 0; n < N; ++n) {
              const float g = to_f32<T>(a[i].e[n]);
              dot = fmaf(g, to_f32<T>(b[i].e[n]), dot);
              o.e[n] = from_f32<T>(wf * g);
            }
            dz[s * V + c0 + i * 32] = o.v;
          }
      }
    }
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, d);
    if (lane == 0) dw[f] = dot;
  }
  zero_tail<VB>(dz, V, R, __ldg(offsets + E), warp_id, num_warps, lane);
}

// The widest vector that divides the row and every base address.
int vec_bytes(int64_t row_bytes, std::initializer_list<const void*> ptrs) {
  uintptr_t bits = static_cast<uintptr_t>(row_bytes);
  for (const void* p : ptrs) bits |= reinterpret_cast<uintptr_t>(p);
  for (int v = 16; v > 1; v >>= 1)
    if (bits % v == 0) return v;
  return 1;
}

int warp_grid(int64_t units) {
  const int64_t blocks = (units + 7) / 8;
  return static_cast<int>(std::max<int64_t>(
      1, std::min<int64_t>(blocks, static_cast<int64_t>(device_sm_count()) * 8)));
}

}  // namespace

size_t expert_sort_smem(int threads, int E) {
  return (static_cast<size_t>(threads / 32) + 2) * (E + 1) * sizeof(int32_t);
}

cudaError_t launch_expert_sort(const int32_t* ids, int64_t R, int E, int32_t* order,
                               int32_t* position, int32_t* offsets, cudaStream_t s,
                               bool keep_dropped) {
  // a slot a thread while 8 CTAs have that many: 8192 slots 5.1 us with 8 CTAs,
  // 5.6 with 4, 6.5 with 2, 9.8 with one; 3111 slots 4.65 with 4, 4.8 with one
  const int threads = R <= 256 ? 256 : 1024;
  int ctas = 1;
  while (ctas < 8 && R > 1024ll * ctas) ctas *= 2;
  const size_t smem = expert_sort_smem(threads, E);
  static DeviceOnce once;
  cudaError_t e = once.run([] {
    return cudaFuncSetAttribute(expert_sort_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                static_cast<int>(expert_sort_smem(1024, kMaxExperts)));
  });
  if (e != cudaSuccess) return e;
  return launch_pdl_cluster(expert_sort_kernel, ctas, threads, smem, ctas, s, ids, R, E, order,
                            position, offsets, keep_dropped);
}

namespace {

// fn(vector width) for the widest vector of rows and bases.
template <typename F>
cudaError_t with_width(int vb, F&& fn) {
  switch (vb) {
    case 16: return fn(std::integral_constant<int, 16>());
    case 8: return fn(std::integral_constant<int, 8>());
    case 4: return fn(std::integral_constant<int, 4>());
    case 2: return fn(std::integral_constant<int, 2>());
    default: return fn(std::integral_constant<int, 1>());
  }
}

constexpr int kGatherU = 4;
int gather_grid(int64_t T, int64_t vecs) {
  return warp_grid(T * ((vecs + kGatherU * 32 - 1) / (kGatherU * 32)));
}

}  // namespace

cudaError_t launch_expert_gather(const void* x, int64_t T, int k, int64_t row_bytes,
                                 const int32_t* position, const int32_t* offsets, int E, void* xs,
                                 cudaStream_t s) {
  return with_width(vec_bytes(row_bytes, {x, xs}), [&](auto width) {
    constexpr int VB = decltype(width)::value;
    using V = typename VecOf<VB>::type;
    const int64_t vecs = row_bytes / VB;
    return launch_pdl(expert_gather_kernel<VB, kGatherU>, gather_grid(T, vecs), 256, 0, s,
                      static_cast<const V*>(x), T, k, vecs, position, offsets, E,
                      static_cast<V*>(xs));
  });
}

cudaError_t launch_expert_dispatch(const void* x, int64_t T, int k, int64_t row_bytes,
                                   const int32_t* ids, int E, int32_t* order, int32_t* position,
                                   int32_t* offsets, void* xs, cudaStream_t s) {
  if (T * k > kDispatchSlots) {
    cudaError_t e = launch_expert_sort(ids, T * k, E, order, position, offsets, s);
    if (e != cudaSuccess) return e;
    return launch_expert_gather(x, T, k, row_bytes, position, offsets, E, xs, s);
  }
  return with_width(vec_bytes(row_bytes, {x, xs}), [&](auto width) {
    constexpr int VB = decltype(width)::value;
    using V = typename VecOf<VB>::type;
    const int64_t vecs = row_bytes / VB;
    const int grid = std::min(gather_grid(T, vecs), device_sm_count());
    return launch_pdl_cluster(expert_dispatch_kernel<VB, kGatherU>, grid, 256,
                              expert_sort_smem(256, E), 1, s, static_cast<const V*>(x), ids, T, k,
                              vecs, E, order, position, offsets, static_cast<V*>(xs));
  });
}

namespace {

// fn(type tag, vector width) for the row type and the widest usable vector;
// narrower than 16 bytes one element at a time.
template <typename T, typename F>
cudaError_t with_vec(int vb, F&& fn) {
  if (vb == 16) return fn(T{}, std::integral_constant<int, 16>());
  return fn(T{}, std::integral_constant<int, sizeof(T)>());
}

template <typename F>
cudaError_t with_type(q8_dtype dt, int vb, F&& fn) {
  switch (dt) {
    case Q8_F32: return with_vec<float>(vb, fn);
    case Q8_F16: return with_vec<__half>(vb, fn);
    default: return with_vec<__nv_bfloat16>(vb, fn);
  }
}

}  // namespace

cudaError_t launch_expert_spread(const void* z, q8_dtype dt, const float* w, int64_t T, int k,
                                 int64_t H, const int32_t* position, void* y, cudaStream_t s) {
  const int64_t row_bytes = H * dtype_bytes(dt);
  return with_type(dt, vec_bytes(row_bytes, {z, y}), [&](auto elem, auto vb) {
    using T_ = decltype(elem);
    constexpr int VB = decltype(vb)::value;
    using V = typename VecOf<VB>::type;
    // (2048 x 4 dispatch and its gradient, 4096 x 8 combine and its: U 2, S 4
    // 34.8 and 137.6 us; 1, 4 39.0 and 147; 4, 2 36.7 and 139.8; 2, 8 37.8 and
    // 138.4; 4, 4 35.7 and 136.8)
    constexpr int U = VB == 16 ? 2 : 4, S = 4;
    const int64_t vecs = row_bytes / VB;
    return launch_pdl(expert_spread_kernel<T_, VB, U, S>,
                      warp_grid(T * ((vecs + U * 32 - 1) / (U * 32))), 256, 0, s,
                      static_cast<const V*>(z), w, T, k, vecs, position, static_cast<V*>(y));
  });
}

cudaError_t launch_expert_combine_bwd(const void* dy, const void* z, q8_dtype dt, const float* w,
                                      int64_t T, int k, int64_t H, const int32_t* position,
                                      const int32_t* offsets, int E, void* dz, float* dw,
                                      cudaStream_t s) {
  const int64_t row_bytes = H * dtype_bytes(dt);
  return with_type(dt, vec_bytes(row_bytes, {dy, z, dz}), [&](auto elem, auto vb) {
    using T_ = decltype(elem);
    constexpr int VB = decltype(vb)::value;
    using V = typename VecOf<VB>::type;
    constexpr int U = VB == 16 ? 2 : 8;
    return launch_pdl(expert_combine_bwd_kernel<T_, VB, U>, warp_grid(T * k), 256, 0, s,
                      static_cast<const V*>(dy), static_cast<const V*>(z), w, T * k, k,
                      row_bytes / VB, position, offsets, E, static_cast<V*>(dz), dw);
  });
}

}  // namespace q8
