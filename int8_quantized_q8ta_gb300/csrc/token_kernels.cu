// token_kernels.cu -- rows with a scale for each token: float rows to int8 and
// back, the operands of the gradients, and the packing of gated weights.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cfloat>
#include <cstdint>
#include <type_traits>

#include "tile_device.cuh"
#include "token_device.cuh"
#include "token_internal.h"
#include "token_split.h"

namespace q8 {

namespace {

// ---------------------------------------------------------------------------
// a = max |x[m]|, s = a / 127, q = rint(x * (1 / s)): a row twice, once for its
// largest magnitude and once to round it.  A CTA has one row at a time and keeps
// it in registers in between, with the next row's loads already on their way; so
// it comes from memory once, and memory is never idle while a row waits for its
// scale.  Only rows beyond U items for each of 704 threads are read again (from
// L2).  Bytes bound it: 8192 rows of 11008 bf16 45 us (floor 41), of 8191 48 (30).
//   SHORT: rows of which a warp holds all items go to a warp each, without a
// barrier (16,000 rows of 200 f16, cold, 6.9 us, 13.2 by CTAs; of 201 13.3, 29).
//   Rows that are no multiple of 8 begin t values into their first item.  q, whose
// rows begin the same way, takes whole items too, but the operand has its own:
// 8 - t values of an item and t of the next one, which a lane gets from the lane
// after it (so a warp's last lane only lends).
// ---------------------------------------------------------------------------
constexpr int kQuantizeThreads = 704;   // at most: two rows' items want some 90 registers
template <int DT>
constexpr int quantize_items() {        // of a thread, in registers
  return DT == Q8_F32 ? 2 : 4;
}

template <int DT, bool VEC, bool OP, bool SHORT>
__global__ void __launch_bounds__(SHORT ? 256 : kQuantizeThreads)
    quantize_token_kernel(const QuantizeJob job) {
  using Rows = FlatRows<DT, VEC>;
  using Item = typename Rows::Item;
  using Lanes = RowLanes<VEC, OP>;
  constexpr int U = quantize_items<DT>();
  __shared__ uint32_t tops[2][32];
  pdl_wait();
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31;
  // this row's warps, and which of them this is; rows on their way at once
  const int warp = SHORT ? 0 : threadIdx.x >> 5, warps = SHORT ? 1 : blockDim.x >> 5;
  const int64_t teams = SHORT ? blockDim.x >> 5 : 1;   // rows of a CTA
  const int64_t m0 = blockIdx.x * teams + (SHORT ? threadIdx.x >> 5 : 0);
  const int64_t m_step = gridDim.x * teams;
  if constexpr (OP)
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
         i < job.count_words; i += static_cast<int64_t>(gridDim.x) * blockDim.x)
      job.counts[i] = 0;
  const Rows rows(job.x, job.M, job.K);
  const bool q_whole = (reinterpret_cast<uintptr_t>(job.q) - rows.off) % 8 == 0;
  const int chunks = job.KB * 8;   // of the operand's row
  // this thread's items: every step'th, of those that whole warps go through
  const int c0 = Lanes::first(warp, lane), step = Lanes::step(warps);
  const int items = Lanes::items(rows.K, chunks);
  Item held[U];
  typename Rows::Row row = rows.row(m0);
#pragma unroll
  for (int u = 0; u < U; ++u) rows.load(held[u], row, c0 + u * step);
  int turn = 0;
  for (int64_t m = m0; m < job.M; m += m_step, turn ^= 1) {
    Item next[U];
    const typename Rows::Row next_row = rows.row(m + m_step);
#pragma unroll
    for (int u = 0; u < U; ++u) rows.load(next[u], next_row, c0 + u * step);
    // (items beyond those: at least in L2 when their row comes)
    for (int c = c0 + U * step; c * 8 < next_row.hi; c += step) prefetch_l2(next_row.at + c * 8);
    uint32_t top = 0;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      rows.settle(held[u], row, c0 + u * step);
      top = max(top, held[u].top());
    }
    for (int c = c0 + U * step; c * 8 - row.t < rows.K; c += step) {
      Item it;
      rows.load(it, row, c);
      rows.settle(it, row, c);
      top = max(top, it.top());
    }
    top = __reduce_max_sync(0xffffffffu, top);
    if constexpr (!SHORT) {
      if (lane == 0) tops[turn][warp] = top;
      __syncthreads();
      top = __reduce_max_sync(0xffffffffu, lane < warps ? tops[turn][lane] : 0u);
    }
    const TokenScale sc = token_scale(top);
    if (warp == 0 && lane == 0) job.scales[m] = sc.scale;
    int8_t* q_row = job.q == nullptr ? nullptr : job.q + m * job.K;
    const auto put = [&](const Item& it, int c) {
      const uint2 q = it.quantize(sc.inv);
      const int e = c * 8 - row.t;
      if (q_row != nullptr && Lanes::stores(lane)) {
        int8_t* to = q_row + e;
        if (VEC ? e < rows.K : q_whole && e >= 0 && e + 8 <= rows.K) {
          *reinterpret_cast<uint2*>(to) = q;
        } else if (!VEC) {
#pragma unroll
          for (int j = 0; j < 8; ++j)
            if (e + j >= 0 && e + j < rows.K)
              to[j] = static_cast<int8_t>((j < 4 ? q.x : q.y) >> (8 * (j & 3)));
        }
      }
      if constexpr (OP) {
        uint2 own = q;
        if constexpr (!VEC) {
          const uint32_t x2 = __shfl_down_sync(0xffffffffu, q.x, 1);
          const uint32_t y2 = __shfl_down_sync(0xffffffffu, q.y, 1);
          const int bits = (row.t & 3) * 8;   // (an item's own from byte t on)
          own = row.t < 4
                    ? make_uint2(__funnelshift_r(q.x, q.y, bits), __funnelshift_r(q.y, x2, bits))
                    : make_uint2(__funnelshift_r(q.y, x2, bits), __funnelshift_r(x2, y2, bits));
        }
        if (c < chunks && Lanes::stores(lane))
          *reinterpret_cast<uint4*>(job.operand + ((c >> 3) * job.M + m) * 64 + (c & 7) * 8) =
              token_f16x8(own);
      }
    };
    // (whole warps go through, for the shuffles)
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (c0 + u * step - lane < items) put(held[u], c0 + u * step);
    for (int c = c0 + U * step; c - lane < items; c += step) {
      Item it;
      rows.load(it, row, c);
      rows.settle(it, row, c);
      put(it, c);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) held[u] = next[u];
    row = next_row;
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

// out = float(q) * s, one rounding to the type.  Items of 8 values on 8 (q) and
// 16 (out) bytes: rows that are no multiple of 8 begin inside an item, which
// both rows take, each its own values of it.  ANY: q or out lie on other bytes,
// one value an item.
template <int DT, bool ANY>
__global__ void __launch_bounds__(256) dequantize_token_kernel(const int8_t* q,
                                                               const float* scales, int64_t M,
                                                               int64_t K, void* out) {
  constexpr int U = 4;
  pdl_wait();
  pdl_launch_dependents();
  if constexpr (ANY) {
    warp_segments<U>(M, K, [&](int64_t m, int64_t c0) {
      const float s = scales[m];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int64_t i = m * K + c0 + u * 32;
        if (c0 + u * 32 < K) store_one<DT>(out, i, __fmul_rn(static_cast<float>(q[i]), s));
      }
    });
  } else {
    const int64_t whole = M * K / 8 * 8;   // items from there on end the rows
    const int64_t items = K % 8 == 0 ? K / 8 : K / 8 + 2;
    warp_segments<U>(M, items, [&](int64_t m, int64_t c0) {
      const float s = scales[m];
      const int64_t row = m * K, first = (row / 8 + c0) * 8;
      uint2 w[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int64_t i = first + u * 256;
        if (i < whole && i < row + K) w[u] = __ldcs(reinterpret_cast<const uint2*>(q + i));
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int64_t i = first + u * 256;
        if (i < whole && i >= row && i + 8 <= row + K) {
          float v[8];
#pragma unroll
          for (int j = 0; j < 8; ++j)
            v[j] = __fmul_rn(
                static_cast<float>(static_cast<int8_t>((j < 4 ? w[u].x : w[u].y) >> (8 * (j & 3)))),
                s);
          store_x8<DT>(out, i, v);
        } else {
#pragma unroll 1
          for (int64_t j = max(i, row); j < min(i + 8, row + K); ++j)
            store_one<DT>(out, j, __fmul_rn(static_cast<float>(q[j]), s));
        }
      }
    });
  }
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

// A CTA has one row at a time in registers, 8 values an item and up to 4
// items a thread (longer rows are read a second time), its items' scales with them for
// all its rows, and the next row's loads on their way.  With wn = ws over the
// power of two of the largest, |dy * wn| < 2 a.
template <bool VEC, bool MASK>
constexpr int grad_items() {   // of a thread, in registers
  return VEC && !MASK ? 4 : VEC || !MASK ? 2 : 1;
}

template <int DT, bool VEC, bool MASK>
__global__ void __launch_bounds__(512) grad_operand_kernel(const GradOperandJob job) {
  constexpr int U = grad_items<VEC, MASK>();
  __shared__ uint32_t slots[3][32];
  pdl_wait();
  pdl_launch_dependents();
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
       i < job.count_words; i += static_cast<int64_t>(gridDim.x) * blockDim.x)
    job.counts[i] = 0;
  const int64_t items = static_cast<int64_t>(job.KB) * 8;
  using Item = RowItem<4, VEC>;
  constexpr int V = MASK ? 2 : 1;   // dy, y
  const int64_t bytes = job.N * 2;
  const bool ws16 = reinterpret_cast<uintptr_t>(job.ws) % 16 == 0;
  const auto load_ws = [&](int64_t c, float (&ws)[8]) {
    if (ws16 && c * 8 + 8 <= job.N) {
      const float4 a = __ldg(reinterpret_cast<const float4*>(job.ws + c * 8));
      const float4 b = __ldg(reinterpret_cast<const float4*>(job.ws + c * 8) + 1);
      const float all[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
      for (int j = 0; j < 8; ++j) ws[j] = all[j];
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) ws[j] = c * 8 + j < job.N ? __ldg(job.ws + c * 8 + j) : 0.0f;
    }
  };
  const auto load = [&](Item (&it)[V], int64_t m, int64_t c) {
    const int64_t n = m < job.M ? bytes : 0;
    it[0].load(row_bytes<uint16_t>(job.dy, job.M, job.N, m), c, n);
    if constexpr (MASK) it[1].load(row_bytes<uint16_t>(job.y, job.M, job.N, m), c, n);
  };
  const auto settle = [&](Item (&it)[V], int64_t m, int64_t c) {
    it[0].settle(row_bytes<uint16_t>(job.dy, job.M, job.N, m), c, bytes);
    if constexpr (MASK) {
      it[1].settle(row_bytes<uint16_t>(job.y, job.M, job.N, m), c, bytes);
#pragma unroll
      for (int j = 0; j < 4; ++j) it[0].w[j] &= above_zero<DT>(it[1].w[j]);
    }
  };
  const auto load_row = [&](Item (&held)[U][V], int64_t m) {
#pragma unroll
    for (int u = 0; u < U; ++u) load(held[u], m, threadIdx.x + static_cast<int64_t>(u) * blockDim.x);
  };
  const auto top16 = [&](const Item& it) {
    const uint32_t t = __vmaxu2(__vmaxu2(it.w[0] & 0x7fff7fffu, it.w[1] & 0x7fff7fffu),
                                __vmaxu2(it.w[2] & 0x7fff7fffu, it.w[3] & 0x7fff7fffu));
    return magnitude(half_bits_to_float<DT>(max(t & 0xffffu, t >> 16)));
  };
  Item held[U][V];
  float held_ws[U][8];
  load_row(held, blockIdx.x);
  uint32_t ws_top = 0;
#pragma unroll
  for (int u = 0; u < U; ++u) load_ws(threadIdx.x + static_cast<int64_t>(u) * blockDim.x, held_ws[u]);
#pragma unroll
  for (int u = 0; u < U; ++u)
#pragma unroll
    for (int j = 0; j < 8; ++j) ws_top = max(ws_top, magnitude(held_ws[u][j]));
  const int64_t held_to = static_cast<int64_t>(U) * 8 * blockDim.x;
  if (held_to < job.N) ws_top = max(ws_top, top_of(job.ws + held_to, job.N - held_to));
  // (a power of two of the largest scale in [1, 2))
  const RowPower channel = row_power(__uint_as_float(block_max(ws_top, slots[2])));
  const float to_one = channel.rescale * 0x1p-14f, from_one = channel.unscale * 0x1p14f;
#pragma unroll
  for (int u = 0; u < U; ++u)
#pragma unroll
    for (int j = 0; j < 8; ++j) held_ws[u][j] *= to_one;
  const auto put = [&](int64_t m, int64_t c, const Item& it, const float (&ws)[8], float rescale) {
    const auto& d = it.w;
    uint32_t r[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
      r[j] = grad_bits_x2(half_bits_to_float<DT>(d[j] & 0xffffu) * rescale * ws[2 * j],
                          half_bits_to_float<DT>(d[j] >> 16) * rescale * ws[2 * j + 1]);
    *reinterpret_cast<uint4*>(job.dst + ((c >> 3) * job.M + m) * 64 + (c & 7) * 8) =
        make_uint4(r[0], r[1], r[2], r[3]);
  };
  int turn = 0;
  for (int64_t m = blockIdx.x; m < job.M; m += gridDim.x, turn ^= 1) {
    Item next[U][V];
    load_row(next, m + gridDim.x);
    uint32_t top = 0;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      settle(held[u], m, threadIdx.x + static_cast<int64_t>(u) * blockDim.x);
      top = max(top, top16(held[u][0]));
    }
    for (int64_t c = threadIdx.x + static_cast<int64_t>(U) * blockDim.x; c < items; c += blockDim.x) {
      Item it[V];
      load(it, m, c);
      settle(it, m, c);
      top = max(top, top16(it[0]));
    }
    // the row's largest between 2^13 and 2^14, times |wn| < 2 (twice the largest
    // would be no number for bf16's largest); rows of subnormal numbers as if they
    // reached the normal ones
    const RowPower row =
        row_power(__uint_as_float(max(block_max(top, slots[turn]), magnitude(FLT_MIN))), 13);
    if (threadIdx.x == 0) job.unscale[m] = row.unscale * from_one;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t c = threadIdx.x + static_cast<int64_t>(u) * blockDim.x;
      if (c < items) put(m, c, held[u][0], held_ws[u], row.rescale);
    }
    for (int64_t c = threadIdx.x + static_cast<int64_t>(U) * blockDim.x; c < items;
         c += blockDim.x) {
      float ws[8];
      load_ws(c, ws);
#pragma unroll
      for (int j = 0; j < 8; ++j) ws[j] *= to_one;
      Item it[V];
      load(it, m, c);
      settle(it, m, c);
      put(m, c, it[0], ws, row.rescale);
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int v = 0; v < V; ++v) held[u][v] = next[u][v];
  }
}

// What the gated gradient's kernel reads beside the weights: the int8 rows as its
// operand, each row's largest |dh|, and from the first four CTAs the largest
// scales and biases, one each.  A row's loads are all in flight before any is used.
template <int DT, bool VEC_Q, bool VEC_DH>
__global__ void __launch_bounds__(512, 3) gated_grad_front_kernel(const GatedGradFrontJob job) {
  constexpr int UD = 4, UQ = 2;
  __shared__ uint32_t slots[2][32];
  pdl_wait();
  pdl_launch_dependents();
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
       i < job.count_words; i += static_cast<int64_t>(gridDim.x) * blockDim.x)
    job.counts[i] = 0;
  if (blockIdx.x < 4) {   // of the gate's and the up projection's scales, and of their biases
    const int i = blockIdx.x;
    const float* v = i < 2 ? job.ws : job.bias;
    const uint32_t top =
        v == nullptr ? 0u : block_max(top_of(v + (i & 1) * job.N, job.N), slots[0]);
    if (threadIdx.x == 0) job.tops[i] = __uint_as_float(top);
    return;
  }
  const FlatRows<DT, VEC_DH> dh(job.dh, job.M, job.N);
  const int items = static_cast<int>((job.N + 14) / 8);
  const int64_t chunks = static_cast<int64_t>(job.KB) * 8;
  const int8_t* q_end = job.q + job.M * job.K;
  int turn = 0;
  for (int64_t m = blockIdx.x - 4; m < job.M; m += gridDim.x - 4, turn ^= 1) {
    uint32_t t = 0;
    const auto row = dh.row(m);
#pragma unroll 1
    for (int c0 = threadIdx.x; c0 < items; c0 += UD * blockDim.x) {
      typename FlatRows<DT, VEC_DH>::Item it[UD];
#pragma unroll
      for (int u = 0; u < UD; ++u)
        dh.load(it[u], row, c0 + u * blockDim.x);
#pragma unroll
      for (int u = 0; u < UD; ++u) {
        dh.settle(it[u], row, c0 + u * blockDim.x);
#pragma unroll
        for (int j = 0; j < 4; ++j) t = __vmaxu2(t, it[u].w[j] & 0x7fff7fffu);
      }
    }
#pragma unroll 1
    for (int64_t c0 = threadIdx.x; c0 < chunks; c0 += static_cast<int64_t>(UQ) * blockDim.x) {
      uint2 w[UQ];
#pragma unroll
      for (int u = 0; u < UQ; ++u)
        w[u] = load_int8x8<VEC_Q>(job.q, m * job.K,
                                  (c0 + static_cast<int64_t>(u) * blockDim.x) * 8, job.K, q_end);
#pragma unroll
      for (int u = 0; u < UQ; ++u) {
        const int64_t c = c0 + static_cast<int64_t>(u) * blockDim.x;
        if (c < chunks)
          *reinterpret_cast<uint4*>(job.operand + ((c >> 3) * job.M + m) * 64 + (c & 7) * 8) =
              token_f16x8(w[u]);
      }
    }
    const uint32_t most =
        block_max(magnitude(half_bits_to_float<DT>(max(t & 0xffffu, t >> 16))), slots[turn]);
    if (threadIdx.x == 0) job.most_dh[m] = __uint_as_float(most);
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
    uint32_t v[4] = {0, 0, 0, 0};
    if constexpr (T) {
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        const int64_t pair = in0 + j;   // the interleaved index
        const int64_t n = (pair >> 5) * 16 + (pair & 15);
        if (n < N && row < K)
          v[j / 4] |= static_cast<uint32_t>(
                          static_cast<uint8_t>(((pair & 16) ? up : gate)[n * K + row]))
                      << (8 * (j % 4));
      }
    } else {
      const int64_t n = (row >> 5) * 16 + (row & 15);
      const int8_t* w = (row & 16) ? up : gate;
      if (n < N) {
        const uint2 a = load_int8x8<false>(w, n * K, in0, K, w + N * K);
        const uint2 b = load_int8x8<false>(w, n * K, in0 + 8, K, w + N * K);
        v[0] = a.x;
        v[1] = a.y;
        v[2] = b.x;
        v[3] = b.y;
      }
    }
    dst[i] = make_uint4(v[0] ^ 0x80808080u, v[1] ^ 0x80808080u, v[2] ^ 0x80808080u,
                        v[3] ^ 0x80808080u);
  }
}

bool on16(const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }

int blocks_for(int64_t warps) {
  return static_cast<int>(std::max<int64_t>(
      1, std::min<int64_t>((warps + 7) / 8, static_cast<int64_t>(device_sm_count()) * 8)));
}

// CTAs of so many threads that an SM takes at once, asked for once each (`fit`, by
// warps): a persistent kernel's rows are dealt to those, and a second wave of CTAs
// would only wait for the first (4096 rows of 4096 f32 16.6 us, 14.7 without).
template <typename K>
int64_t resident_ctas(K kernel, int threads, std::atomic<int> (&fit)[33]) {
  int n = fit[threads / 32].load(std::memory_order_relaxed);
  if (n == 0) {
    if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kernel, threads, 0) != cudaSuccess || n < 1) {
      cudaGetLastError();
      n = 1;
    }
    fit[threads / 32].store(n, std::memory_order_relaxed);
  }
  return n;
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
  // else as many as it holds, and as many CTAs as the SMs take at once.
  const int K = static_cast<int>(job.K), chunks = job.KB * 8;
  const int64_t items = job.operand != nullptr ? (vec ? RowLanes<true, true>::items(K, chunks)
                                                      : RowLanes<false, true>::items(K, chunks))
                        : vec                  ? RowLanes<true, false>::items(K, chunks)
                                               : RowLanes<false, false>::items(K, chunks);
  const int held = dtype == Q8_F32 ? quantize_items<Q8_F32>() : quantize_items<Q8_F16>();
  const int64_t lanes =
      job.operand != nullptr && !vec ? RowLanes<false, true>::kStoring : RowLanes<true, true>::kStoring;
  const bool few = job.M <= 2 * device_sm_count();
  const auto go = [&](auto t, auto v, auto s_) {
    constexpr int DT = decltype(t)::value;
    constexpr bool VEC = decltype(v)::value, SHORT = decltype(s_)::value;
    int64_t threads = 256, rows = 8;   // of a CTA
    if constexpr (!SHORT) {
      const int64_t each = few ? 1 : held;
      threads = 32 * std::min<int64_t>(kQuantizeThreads / 32,
                                       std::max<int64_t>(2, (items + each * lanes - 1) / (each * lanes)));
      rows = 1;
    }
    const auto launch = [&](auto kernel, std::atomic<int>(&fit)[33]) {
      const int64_t ctas = resident_ctas(kernel, static_cast<int>(threads), fit) * device_sm_count();
      const int grid = static_cast<int>(std::min<int64_t>((job.M + rows - 1) / rows, ctas));
      return launch_pdl(kernel, grid, static_cast<int>(threads), 0, s, job);
    };
    static std::atomic<int> fit[2][33];
    return job.operand != nullptr ? launch(quantize_token_kernel<DT, VEC, true, SHORT>, fit[0])
                                  : launch(quantize_token_kernel<DT, VEC, false, SHORT>, fit[1]);
  };
  const bool is_short = !few && items <= held * lanes;
  return by_type(dtype, vec, [&](auto t, auto v) {
    return is_short ? go(t, v, std::true_type()) : go(t, v, std::false_type());
  });
}

cudaError_t launch_dequantize_token(const int8_t* q, const float* scales, int64_t M, int64_t K,
                                    q8_dtype dtype, void* out, cudaStream_t s) {
  const bool any = !on16(out) || reinterpret_cast<uintptr_t>(q) % 8 != 0;
  const int64_t items = any ? K : K % 8 == 0 ? K / 8 : K / 8 + 2;
  const int grid = blocks_for(M * ((items + 127) / 128));
  return by_type(dtype, any, [&](auto t, auto v) {
    return launch_pdl(dequantize_token_kernel<decltype(t)::value, decltype(v)::value>, grid, 256, 0,
                      s, q, scales, M, K, out);
  });
}

cudaError_t launch_grad_operand(const GradOperandJob& job, q8_dtype dtype, cudaStream_t s) {
  const bool vec = job.N % 8 == 0 && on16(job.dy) && on16(job.y);
  const int64_t items = static_cast<int64_t>(job.KB) * 8;
  const int64_t each =
      job.M <= 2 * device_sm_count() ? 1 : vec && !job.y ? 4 : vec || !job.y ? 2 : 1;   // as grad_items
  const int threads = static_cast<int>(
      std::min<int64_t>(512, std::max<int64_t>(64, round_up((items + each - 1) / each, 32))));
  const auto go = [&](auto t, auto v) {
    constexpr int DT = decltype(t)::value;
    constexpr bool VEC = decltype(v)::value;
    const auto launch = [&](auto kernel, std::atomic<int>(&fit)[33]) {
      const int64_t ctas = resident_ctas(kernel, threads, fit) * device_sm_count();
      return launch_pdl(kernel, static_cast<int>(std::min<int64_t>(job.M, ctas)), threads, 0, s, job);
    };
    static std::atomic<int> fit[2][33];
    return job.y != nullptr ? launch(grad_operand_kernel<DT, VEC, true>, fit[0])
                            : launch(grad_operand_kernel<DT, VEC, false>, fit[1]);
  };
  return by_half(dtype, vec, go);
}

cudaError_t launch_gated_grad_front(const GatedGradFrontJob& job, q8_dtype dtype, cudaStream_t s) {
  const bool vec_dh = job.N % 8 == 0 && on16(job.dh);
  const bool vec_q = job.K % 8 == 0 && reinterpret_cast<uintptr_t>(job.q) % 8 == 0;
  // 4 items of dh a thread, and as many CTAs as the SMs take at once
  const int threads = static_cast<int>(
      std::min<int64_t>(512, std::max<int64_t>(256, round_up((job.N + 31) / 32, 32))));
  const int grid = 4 + static_cast<int>(std::min<int64_t>(
                           job.M, static_cast<int64_t>(device_sm_count()) * (1536 / threads)));
  return by_half(dtype, vec_dh, [&](auto t, auto v) {
    constexpr int DT = decltype(t)::value;
    constexpr bool VEC = decltype(v)::value;
    return vec_q ? launch_pdl(gated_grad_front_kernel<DT, true, VEC>, grid, threads, 0, s, job)
                 : launch_pdl(gated_grad_front_kernel<DT, false, VEC>, grid, threads, 0, s, job);
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

}  // namespace q8
