// tile_gemm_kernel.cuh -- the int8-weight contraction on tcgen05 (sm_103a):
// rows of one batch, sorted into groups, each group times its own int8 weight;
// the shared projection with low-rank adapters, which is one group whose
// tiles get an extra term; and, one group each, the products of rows with a
// scale for each token (tile_gemm_token.cu, tile_gemm_grad.cu; see TileForm).
//
//   acc[s, n] = sum_k (x[s, k] - zp) * w[e(s)][n, k]      exact in int32
//   v = ((float)acc * s_in) * ws[e, n] + b[e, n]  (+ delta[s, n])
//   delta[s, n] = sum_j h[s, j] * B[a(s)][n, j]
// then the activation and either the requantization to int8 or one rounding
// to the float output type.
//
// Weights stay int8 in memory (1 byte read per weight, half of the bf16 copy
// the plain linear keeps): a tile of 128 output channels x 64 inputs is one
// contiguous 8 KB run, copied to shared memory in bulk, turned into f16 by four
// or eight warps (a byte permute and half a packed subtraction per value) and put
// into TENSOR MEMORY as the MMA's A operand.  Tokens are the B operand, f16
// copies of x - zp in K-blocked rows that TMA fetches 128-byte swizzled.  So
// weights are on the MMA's M side (always 128 lanes, however few tokens a
// group has) and tokens on N, 16 to 192 of them in steps of 16; the shared
// memory traffic of a k-block is the tokens' tile and 2 bytes per weight.
//
// Exactness: |x - zp| <= a and sum |w| over 64 inputs <= W give f32 sums that
// are exact integers for 2^24 / (a W) k-blocks; such a chunk is then drained
// from TMEM into int32 registers while another accumulator fills.
//
// Work split: whole waves of (tile, output block) units, then the last one to
// two waves' k-blocks as one line cut into equal runs, one per CTA, so that a
// few wide units and many small ones fill the SMs alike.  A unit cut by a run's
// end is summed by whichever of its CTAs comes last, warp by warp, from the int32
// parts the others left in the workspace: integer sums, the same in any order
// (a gradient's f32 ones in the order of their CTAs).  No CTA waits for another.
//
// Adapters: after a unit's k-blocks, its last run multiplies B[a] by the rows'
// h for each adapter the tile holds, into an accumulator of its own: tf32
// MMAs, B exact (f16 and bf16 both fit tf32), h as the sum of two tf32 terms
// (within its last place), rows of other adapters as zeros.  The kernel before
// this one lays h out so, and it comes through the ring like tokens: fetched
// by the converting warps it queued behind the next unit's copies (a round of
// 16 ranks 1,350 cycles, and 2,000 before the first).
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "row_split.h"
#include "rows_internal.h"
#include "tile_device.cuh"
#include "token_device.cuh"

namespace q8 {

namespace {

enum : uint32_t { kErrTileRing = 0x10A, kErrTileAcc = 0x10B, kErrTileOperand = 0x10C };

constexpr int kMaxRing = 12;
constexpr int kTileWBytes = 128 * 64;   // int8 weights of one tile and k-block
constexpr int kFirstConv = 4;           // warps 0 to 3: weights, MMAs, tokens, schedule
constexpr int kTileThreads = 640;
constexpr int kTmemCols = 512;

// What one kernel computes of its sums.
//   kFormBatch      one activation scale for the batch, groups, adapters
//   kFormToken      v = ((float)acc * s[row]) * ws[n] + b[n]
//   kFormGated      act(g) * u, g and u such values of two weights whose rows
//                   come interleaved, 16 of one and 16 of the other: a warp's
//                   lanes hold both of 16 channels, and one shuffle for two
//                   tokens brings them together (lane l takes one token,
//                   l + 16 the other)
//   kFormGatedGrad  the same g and u, then with dh their two gradients, each
//                   times its channel's ws and its row's power of two, in f16:
//                   the operand of the next kernel
//   kFormGrad       such f16 rows times the transposed weight: f32 sums instead
//                   of exact integers, parts added in the order of their CTAs,
//                   the rows' powers of two taken out again
enum TileForm { kFormBatch, kFormToken, kFormGated, kFormGatedGrad, kFormGrad };

// What the kernels before this one write while it may already run (offsets,
// ids, lists, h, output rows) is read with ordinary loads, not as data that is
// constant for the kernel's life.

// The two forms of the kernel.  (Sizes here and below: rows x outputs x inputs.)
//   Wide (tiles of 65 .. 192 rows): a pair of CTAs on neighbouring SMs shares
// a tile through the 2-SM MMA, each with its own 128 output channels and half
// of the rows in its shared memory: 12 KB of tokens and 8 KB of weights from L2
// for a k-block's 384 cycles of MMAs, where one CTA alone needs 32 KB.  Its four
// converting warps take some 250 cycles a stage to wait and announce and 130 a
// k-block to convert, so a stage is two k-blocks: with one they took 500 cycles
// a k-block and the MMAs waited (2048 rows, the pair 11008 x 4096 gated 221 us);
// now the MMAs are what it waits for (202 us, 83% of the tensor pipe's cycles in
// the kernel; then the GPU's power).  8192 rows of 16 experts x 4096 x 4096: 184
// us (195 so); 2048 rows x 11008 x 4096 with 8 adapters of rank 64 152 (161).
//   Narrow (up to 64 rows): one CTA; two k-blocks a stage and twice the
// converting warps, in two groups.  Conversion and the MMAs' issue take some 480
// cycles a stage each.  128 rows of 56 experts x 2048 x 2048: 37.7 us with the
// operand before it, 35.0 at the copy rate; 24 rows x 11008 x 4096 15.0 us; 64
// rows x 11008 x 4096 with 32 adapters of rank 16 24.4 us; one row x 4096 x 4096
// with its adapter 10.5 to 12 us.
template <bool PAIR>
struct Form {
  static constexpr int CG = PAIR ? 2 : 1;
  static constexpr int KD = 2;                     // k-blocks a stage
  // stages of A operands in tensor memory, behind the accumulators
  static constexpr int NAb = PAIR ? 1 : 2, NA = 1 << NAb;
  static constexpr int kConv = PAIR ? 4 : 8;       // converting warps
  static constexpr int kGroups = kConv / 4;        // groups of four take turns
  static constexpr int kEpi = PAIR ? 12 : 8;       // epilogue warps
  static constexpr int kCols = PAIR ? 64 : 32;     // accumulator columns of each
  // Accumulators (a third one while the epilogue's first dot products take
  // longer than two exact chunks: 64 rows x 11008 x 4096 waited 3 us)
  static constexpr int kAcc = PAIR ? 2 : 3;
  static constexpr int kRing = PAIR ? kMaxRing : 6;   // stages at most
  static constexpr int kFirstEpi = kFirstConv + kConv;
  // Registers of a thread by its part, out of kRegs at launch: what spills finds
  // no L1 beside this much shared memory, and waits behind tokens and weights.
  static constexpr int kControlRegs = 56, kConvRegs = 88, kEpiRegs = PAIR ? 112 : 120;
  static constexpr int kRegs = 96;
  static_assert((kControlRegs * kFirstConv + kConvRegs * kConv + kEpiRegs * kEpi) * 32 <=
                    kRegs * kTileThreads,
                "no more than the block was launched with: it would wait for ever");
  static_assert(32 * (kFirstEpi + kEpi) == kTileThreads, "one block size");
  static constexpr int kMaxRows = kCols * kEpi / 4;
  static_assert(kMaxRows == (PAIR ? kMaxTileRows : kMaxNarrowRows), "tile heights");
  // accumulators, A operands, and row by row the adapters' terms
  static_assert(kAcc * kMaxRows + NA * KD * 32 + (PAIR ? 0 : kMaxRows) <= kTmemCols, "TMEM");
  // int32 words of one CTA's part of a unit
  static constexpr int kPart = kEpi * kCols * 32;
  static_assert(kPart <= kTilePartWords, "workspace");
  static_assert(kEpi <= kTileEpiWarps, "workspace");
};

// One run's part of a unit, as the scheduling warp hands it to the others.
struct alignas(16) Seg {
  int e, row0, rows, nb;       // group, first row, rows, output block (of 128 * CG)
  int tile, kb0, kb1;          // index of the row tile; k-blocks; kb1 0: no more
  int na;                      // adapters whose MMAs follow (see adapters_of)
  int first, end;              // CTAs (pairs) that share the unit
  int pad[2];
};
constexpr int kSegs = 4;       // parts on their way

struct TileShared {
  uint64_t wfull[kMaxRing];   // weights of a stage have landed
  uint64_t tfull[kMaxRing];   // tokens of a stage have landed (a pair's halves: at the leader)
  uint64_t empty[kMaxRing];   // a stage's MMAs are done
  uint64_t ready[4];          // A operand in TMEM
  uint64_t acc_full[3];
  uint64_t acc_empty[3];
  uint64_t drain;
  uint64_t seg_full[kSegs];   // a part is described
  uint64_t seg_empty[kSegs];  // every warp has read it
  Seg seg[kSegs];
  uint32_t tmem;
  uint32_t abort;
  int32_t tiles;              // row tiles of all groups
  alignas(16) float corner[kTileEpiWarps][8][16];   // h of the rows a warp is at
};

// Ring stages per exact f32 chunk.
template <int KD, bool FLOAT>
__device__ __forceinline__ int chunk_stages_of(const TileParams& p) {
  if constexpr (FLOAT) return 1 << 28;   // nothing to keep exact
  int wb = __ldg(p.w_bound);
  if (wb < 1 || wb > kWorstWBound) wb = wb < 1 ? 1 : kWorstWBound;
  return max(1, (1 << 24) / (p.a_bound * wb) / KD);
}

// Rows of group e.  Offsets come from device memory: whatever they hold, no
// row outside [0, R) is touched.
__device__ __forceinline__ int group_end(const TileParams& p, int e) {
  return min(p.R, max(0, p.offsets[e]));
}
__device__ __forceinline__ int group_rows(const TileParams& p, int e, int& start) {
  start = group_end(p, e);
  return max(0, group_end(p, e + 1) - start);
}

// The units of a CTA (or pair), a unit being a row tile times 128 (256)
// channels.  While whole waves of units remain, the CTAs take neighbouring
// ones, the row tiles of one output block after another: what runs at the same
// time then shares its weights and tokens in L2 (contiguous runs for each CTA
// kept every expert's weights in flight at once, more than L2 holds).  The
// last one to two waves form a line of k-blocks cut into equal runs; where
// `aligned` (one group) and what the whole waves leave is a quarter wave or more,
// that alone does, so that CTAs stay at the same inputs for as long as they can:
// 1024 rows x 4096 x 22016, whose weights and rows L2 cannot hold, read 657 MB
// of memory for 135 without, 161 us against 152.  (Less than a quarter would be
// cut into more parts than are worth joining: 900 rows x 4096 x 4096, 4 units
// for 76 pairs, 56 us against 38.)
//   (All counts fit 32 bits: the host checks.)
template <int CG>
struct Walk {
  const TileParams& p;
  const int32_t* prefix;   // row tiles before each group, or null: one group
  int NB;                  // blocks of 128 * CG channels
  int ctas, me;            // CTAs (pairs) and this one
  int waves, wave;         // whole waves, and those behind
  int base, q;             // the line's first unit, and k-blocks of a run
  int share;               // CTAs to each of the line's units, where runs end with units; or 0
  int left, unit, kb;      // the run's k-blocks still to take; its unit and where in it
  int e, start, count;     // the unit's group and its rows
  int tiles, per, t0;      // the group's row tiles, rows of each, tiles before them
  int i, nb;               // row tile and output block

  __device__ __forceinline__ Walk(const TileParams& p_, const int32_t* prefix_, int all_tiles,
                                  bool aligned)
      : p(p_), prefix(prefix_), NB((p_.NB + CG - 1) / CG) {
    ctas = gridDim.x / CG;
    me = blockIdx.x / CG;
    const int units = all_tiles * NB, full = units / ctas;
    const int behind = units - full * ctas;
    waves = behind == 0 || (aligned && behind >= ctas / 4) ? full : max(full - 1, 0);
    wave = 0;
    base = waves * ctas;
    const int total = (units - base) * p.KB;
    q = max(p.min_run, (total - 1) / ctas + 1);
    const int rest = units - base, whole = (rest + ctas - 1) / ctas * p.KB;
    const bool few = 2 * rest <= ctas;
    const int join = CG == 2 ? kJoinWide : p.by_row && !few ? kJoinByRow : kJoinNarrow;
    if (whole <= q + join) q = max(whole, 1);
    // Few units: as many CTAs to each as there are, no run across two of them
    // (its CTA would join parts twice)
    share = rest > 0 && few && q < p.KB
                ? max(1, min(ctas / rest, p.KB / max(1, p.min_run)))
                : 0;
    unit = -1;             // the run is not begun
    if (share > 0) {
      const int part = me % share;
      kb = part_start(part, p.KB, share);
      left = me / share < rest ? part_start(part + 1, p.KB, share) - kb : 0;
      return;
    }
    kb = static_cast<int>(min(static_cast<int64_t>(total), static_cast<int64_t>(q) * me));
    left = min(total - kb, q);
  }
  __device__ __forceinline__ void cut() {
    tiles = (count + p.TN - 1) / p.TN;
    per = tile_rows(count, tiles);
  }
  // Divisions and a search, once a whole unit or run.
  __device__ __forceinline__ void locate(int u) {
    e = 0;
    start = 0;
    count = p.R;
    t0 = 0;
    if (prefix != nullptr) {
      // the last group that starts at or before this unit (groups without
      // rows have no units)
      int lo = 0, hi = p.E - 1;
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (prefix[mid] * NB <= u) lo = mid; else hi = mid - 1;
      }
      e = lo;
      t0 = prefix[lo];
      count = group_rows(p, e, start);
    }
    cut();
    const int local = u - t0 * NB;
    nb = local / tiles;
    i = local - nb * tiles;
  }
  __device__ __forceinline__ void fill(Seg& s) const {
    s.e = e;
    s.nb = nb;
    s.row0 = start + i * per;
    s.rows = min(per, count - i * per);
    s.tile = t0 + i;
  }
  __device__ __forceinline__ bool next(Seg& s) {
    if (wave < waves) {
      locate(wave++ * ctas + me);
      fill(s);
      s.kb0 = 0;
      s.kb1 = p.KB;
      s.first = s.end = me;
      return true;
    }
    if (left <= 0) return false;
    if (unit < 0) {   // (the whole waves left other units' places behind)
      const int skip = share > 0 ? me / share : kb / p.KB;
      unit = base + skip;
      if (share == 0) kb -= skip * p.KB;
      locate(unit);
    }
    fill(s);
    s.kb0 = kb;
    s.kb1 = min(p.KB, kb + left);
    if (share > 0) {
      s.first = (unit - base) * share;
      s.end = s.first + share - 1;
    } else {
      s.first = (unit - base) * p.KB / q;
      s.end = ((unit - base + 1) * p.KB - 1) / q;
    }
    left -= s.kb1 - s.kb0;
    if (left > 0) {
      kb = 0;
      ++unit;
      if (++i == tiles) {
        i = 0;
        if (++nb == NB) {
          nb = 0;
          t0 += tiles;
          do {
            ++e;
            count = group_rows(p, e, start);
          } while (count == 0 && e + 1 < p.E);
          cut();
        }
      }
    }
    return true;
  }
};

// A place in the ring and the parity of its current round.
struct Ring {
  int slot = 0;
  uint32_t phase = 0;
  __device__ __forceinline__ void advance(int stages) {
    if (++slot == stages) {
      slot = 0;
      phase ^= 1u;
    }
  }
};

// The parts in turn, for a whole warp; a part stays where it is, in shared
// memory, until the next is asked for.
struct Feed {
  TileShared& sh;
  Ring ring;
  int last = -1;
  __device__ __forceinline__ const Seg* next(volatile uint32_t* abort_flag, uint32_t* err) {
    if (last >= 0) {
      __syncwarp();
      if ((threadIdx.x & 31) == 0) mbar_arrive(smem_u32(&sh.seg_empty[last]));
    }
    last = ring.slot;
    if (!tile_wait_warp(smem_u32(&sh.seg_full[last]), ring.phase, abort_flag, kErrTileRing, err))
      return nullptr;
    ring.advance(kSegs);
    return sh.seg[last].kb1 > 0 ? &sh.seg[last] : nullptr;
  }
};

// Adapters of the unit's rows, where this run holds the unit's end and MMAs
// take them.
__device__ __forceinline__ int adapters_of(const TileParams& p, const Seg& s) {
  return (p.L > 0 && !p.by_row && s.kb1 == p.KB)
             ? p.lists[static_cast<int64_t>(s.tile) * p.list_stride]
             : 0;
}

// sum_j h[s, j] B[a(s)][n, j] for one channel and 8 rows a call, by a whole
// warp: lane u < 8 holds row u's index my_s and adapter my_a (out of range:
// none).  B comes from global memory, 16 bytes a thread, four rows' loads at a
// time; the rows' h, 16 ranks at a time, through the warp's corner of shared
// memory, from where all lanes read the same words.  row: the channel's place
// among its block's 128.
__device__ __forceinline__ void row_deltas(const TileParams& p, int nb, int row, int my_a, int my_s,
                                           float (*corner)[16], float (&d)[8]) {
  const int lane = threadIdx.x & 31;
  const bool mine = my_a >= 0 && my_a < p.L;
  const uint32_t have = __ballot_sync(0xffffffffu, mine);
  const int my_at = mine ? my_a * p.NB + nb : 0;
#pragma unroll
  for (int u = 0; u < 8; ++u) d[u] = 0.0f;
  if (have == 0) return;
  // this lane's quarter of 16 ranks of row lane / 4 (rows without an adapter
  // have no h)
  const bool h_in = (have >> (lane >> 2)) & 1;
  const float4* h = reinterpret_cast<const float4*>(
      p.h + static_cast<int64_t>(__shfl_sync(0xffffffffu, my_s, lane >> 2)) * p.rank16 * 16);
  for (int c = 0; c < p.rank16; ++c) {
    const float4 hv = h_in ? h[c * 4 + (lane & 3)] : make_float4(0.f, 0.f, 0.f, 0.f);
    __syncwarp();
    *reinterpret_cast<float4*>(&corner[lane >> 2][(lane & 3) * 4]) = hv;
    __syncwarp();
#pragma unroll
    for (int u0 = 0; u0 < 8; u0 += 4) {
      uint4 v[4][2];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int64_t at = __shfl_sync(0xffffffffu, my_at, u0 + u);
        const uint8_t* b = p.lora_b + (at * p.rank16 + c) * 4096 + row * 16;
#pragma unroll
        for (int g = 0; g < 2; ++g)
          v[u][g] = (have >> (u0 + u)) & 1
                        ? __ldg(reinterpret_cast<const uint4*>(b + g * 2048))
                        : make_uint4(0, 0, 0, 0);
      }
#pragma unroll
      for (int u = 0; u < 4; ++u)
#pragma unroll
        for (int g = 0; g < 2; ++g) {
          const float4 h0 = *reinterpret_cast<const float4*>(&corner[u0 + u][g * 8]);
          const float4 h1 = *reinterpret_cast<const float4*>(&corner[u0 + u][g * 8 + 4]);
          const uint32_t q[4] = {v[u][g].x, v[u][g].y, v[u][g].z, v[u][g].w};
          const float f[8] = {h0.x, h0.y, h0.z, h0.w, h1.x, h1.y, h1.z, h1.w};
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            float2 w;
            if (p.lora_f16) {
              w = __half22float2(*reinterpret_cast<const __half2*>(&q[j]));
            } else {
              w.x = __uint_as_float(q[j] << 16);
              w.y = __uint_as_float(q[j] & 0xffff0000u);
            }
            d[u0 + u] = fmaf(f[j * 2], w.x, d[u0 + u]);
            d[u0 + u] = fmaf(f[j * 2 + 1], w.y, d[u0 + u]);
          }
        }
    }
  }
}

// v of one accumulator without its adapter term, in the order of the header's
// epilogue.
__device__ __forceinline__ float dequant(int32_t acc, float ws, float b, const Requant& rq) {
  float t = __fmul_rn(__int2float_rn(acc), rq.s_in);
  t = __fmul_rn(t, ws);
  return __fadd_rn(t, b);
}

// One word of another CTA's part.
template <bool FLOAT>
__device__ __forceinline__ void add_part(int32_t& acc, int32_t v) {
  if constexpr (FLOAT) acc = __float_as_int(__fadd_rn(__int_as_float(acc), __int_as_float(v)));
  else acc += v;
}

template <int OUT> struct OutType { using type = uint16_t; };
template <> struct OutType<Q8_I8> { using type = int8_t; };
template <> struct OutType<Q8_F32> { using type = float; };

// An output's last step: requantize, or activate and round.
template <int OUT>
__device__ __forceinline__ typename OutType<OUT>::type finish(float v, const TileParams& p) {
  if constexpr (OUT == Q8_I8) {
    return static_cast<int8_t>(round_clamp_first(__fmul_rn(v, p.rq.inv_out), p.rq.ozp_i, p.rq.lo_f,
                                                 p.rq.hi_f));
  } else {
    v = max_nan(v, p.floor_f);   // relu: floor 0, else -inf
    if constexpr (OUT == Q8_F32) return v;
    else if constexpr (OUT == Q8_F16) return __half_as_ushort(__float2half_rn(v));
    else return __bfloat16_as_ushort(__float2bfloat16_rn(v));
  }
}

// What the epilogue of rows with a scale for each token wants beside the sums,
// asked for while the MMAs run: a warp's 32 channels and `mine` columns from
// col0 on of one unit (lane l: channel l, columns l and l + 32).
template <TileForm FORM>
struct TokenScales {
  static constexpr bool kPairs = FORM == kFormGated || FORM == kFormGatedGrad;
  float s0, s1, ws, bias;   // the rows' (of a gradient what undoes their power), the channel's
  float r0, r1;             // the gated gradient: its rows' powers of two
  __device__ __forceinline__ void load(const TileParams& p, const Seg& sg, int nb, int quarter,
                                       int col0, int mine) {
    const int lane = threadIdx.x & 31;
    const int row = nb * 128 + quarter * 32 + lane;   // of the packed weight
    const int n = kPairs ? (row >> 5) * 16 + (lane & 15) : row;
    const int64_t en = (kPairs && (lane & 16) ? static_cast<int64_t>(p.N) : 0) + n;
    ws = bias = s0 = s1 = r0 = r1 = 0.0f;
    if (FORM != kFormGrad && n < p.N) {
      ws = __ldg(p.ws + en);
      if (p.bias != nullptr) bias = __ldg(p.bias + en);
    }
    // (the kernel before this one may have written the rows': ordinary loads)
    const int at = sg.row0 + col0;
    const bool in0 = lane < mine, in1 = lane + 32 < mine;
    const float* rows = FORM == kFormGrad ? p.unscale : p.row_scale;
    if (in0) s0 = rows[at + lane];
    if (in1) s1 = rows[at + lane + 32];
    if constexpr (FORM == kFormGatedGrad) {
      const float4 tops = *reinterpret_cast<const float4*>(p.tops);
      const bool once = nb == 0 && quarter == 0;   // a row's sums' power of two
      if (in0) {
        const RowPower power = gated_row_power(p.most_dh[at + lane], s0, p.K, tops);
        r0 = power.rescale;
        if (once) p.unscale[at + lane] = power.unscale;
      }
      if (in1) {
        const RowPower power = gated_row_power(p.most_dh[at + lane + 32], s1, p.K, tops);
        r1 = power.rescale;
        if (once) p.unscale[at + lane + 32] = power.unscale;
      }
    }
  }
};

// That epilogue, B columns a round.  Rounds stay rolled and the registers move up
// instead: a CTA runs them once to a few times, so their code costs more to fetch
// than to execute, and columns without rows are left out.  my_dh: the gated
// gradient's 16 channels of each column, in shared memory.
template <int OUT, int COLS, TileForm FORM>
__device__ __forceinline__ void token_epilogue(const TileParams& p, const Seg& sg,
                                               int32_t (&acc)[COLS], const TokenScales<FORM>& sc,
                                               int nb, int quarter, int col0, int mine,
                                               const uint16_t* my_dh) {
  using T = typename OutType<OUT>::type;
  constexpr bool kPairs = TokenScales<FORM>::kPairs;
  constexpr int B = 16;
  const int lane = threadIdx.x & 31;
  const int row = nb * 128 + quarter * 32 + lane;   // of the packed weight
  const bool up = kPairs && (lane & 16);
  const int mine_j = up ? 1 : 0;   // gate lanes take tokens j, up lanes j + 1
  const int n = kPairs ? (row >> 5) * 16 + (lane & 15) : row;
  const bool in = n < p.N;
  const int at = sg.row0 + col0;
  // the gated gradient: its operand K-blocked, in the order of the packed rows, 64
  // a block (the block that an odd count repeats for a pair has no place there)
  const float ws_other = kPairs ? __shfl_xor_sync(0xffffffffu, sc.ws, 16) : 0.0f;
  const float wg = up ? ws_other : sc.ws, wu = up ? sc.ws : ws_other;
  const int rows = (FORM == kFormGatedGrad ? nb < p.NB : in) ? mine - mine_j : 0;
  T* out = static_cast<T*>(p.out) + static_cast<int64_t>(at + mine_j) * p.N + n;
  uint16_t* to = p.operand_out +
                 ((static_cast<int64_t>(nb) * 2 + (quarter >> 1)) * p.R + at + mine_j) * 64 +
                 (quarter & 1) * 32 + (lane & 15);
  const uint16_t* dh = my_dh + mine_j * 16 + (lane & 15);
#pragma unroll 1
  for (int j0 = 0; j0 < mine; j0 += B) {
    const float s_of = j0 < 32 ? sc.s0 : sc.s1, r_of = j0 < 32 ? sc.r0 : sc.r1;
#pragma unroll
    for (int j = 0; j < B; ++j) {
      const float s = __shfl_sync(0xffffffffu, s_of, (j0 + j) & 31);
      acc[j] = __float_as_int(FORM == kFormGrad ? __fmul_rn(__int_as_float(acc[j]), s)
                                                : token_value(acc[j], s, sc.ws, sc.bias));
    }
    if constexpr (!kPairs) {
#pragma unroll
      for (int j = 0; j < B; ++j, out += p.N)
        if (j0 + j < rows) *out = finish<OUT>(__int_as_float(acc[j]), p);
    } else {
#pragma unroll
      for (int j = 0; j < B; j += 2) {
        // gate lanes keep token j and send their token j + 1; up lanes the reverse
        const float a = __int_as_float(acc[j]), b = __int_as_float(acc[j + 1]);
        const float other = __shfl_xor_sync(0xffffffffu, up ? a : b, 16);
        const float g = up ? other : a, u = up ? b : other;
        float slope;
        if constexpr (FORM == kFormGated) {
          const float h = activate<false, OUT == Q8_F32>(g, p.act, slope) * u;
          if (j0 + j < rows) *out = finish<OUT>(h, p);
          out += 2 * static_cast<int64_t>(p.N);
        } else {
          const float t = activate<true, false>(g, p.act, slope);
          const float r = __shfl_sync(0xffffffffu, r_of, ((j0 + j) & 31) + mine_j);
          const float v = half_bits_to_float<OUT>(dh[(j0 + j) * 16]) * r;
          // channels past the last hold zeros, whatever the rows' scales are
          const uint32_t both = in ? grad_bits_x2(v * u * slope * wg, v * t * wu) : 0;
          if (j0 + j < rows) {
            to[(j0 + j) * 64] = static_cast<uint16_t>(both);
            to[(j0 + j) * 64 + 16] = static_cast<uint16_t>(both >> 16);
          }
        }
      }
    }
#pragma unroll
    for (int j = 0; j < COLS - B; ++j) acc[j] = acc[j + B];
  }
}

// A warpgroup's registers from here on.
template <int N>
__device__ __forceinline__ void split_registers() {
  if constexpr (N < Form<true>::kRegs) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
  else asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}

// Two halves of a token tile have rows that are multiples of 8.
template <int OUT, bool PAIR, TileForm FORM>
__global__ void __launch_bounds__(kTileThreads, 1)
    tile_gemm_kernel(const __grid_constant__ CUtensorMap map_x,
                     const __grid_constant__ CUtensorMap map_h, const TileParams p) {
  using F = Form<PAIR>;
  constexpr int CG = F::CG, KD = F::KD, NAb = F::NAb, NA = F::NA, kCols = F::kCols;
  constexpr bool kBatch = FORM == kFormBatch, kFloat = FORM == kFormGrad;
  extern __shared__ __align__(1024) uint8_t dyn[];
  __shared__ TileShared sh;
  const int warp = uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;
  const int rank = PAIR ? static_cast<int>(cluster_ctarank()) : 0;
  const bool leader = rank == 0;
  const uint32_t ring0 = (smem_u32(dyn) + 1023u) & ~1023u;
  const int S = p.stages;
  const uint32_t acc_cols = p.TN;
  const uint32_t tok_bytes = static_cast<uint32_t>(p.TN / CG) * 128u;
  const uint32_t stage_bytes = static_cast<uint32_t>(KD) * (tok_bytes + kTileWBytes);
  int32_t* prefix = kBatch && p.offsets != nullptr
                        ? reinterpret_cast<int32_t*>(dyn + (ring0 - smem_u32(dyn)) +
                                                     static_cast<size_t>(S) * stage_bytes)
                        : nullptr;

  if (threadIdx.x == 0) {
    for (int i = 0; i < S; ++i) {
      mbar_init(smem_u32(&sh.wfull[i]), 1);
      mbar_init(smem_u32(&sh.tfull[i]), 1);
      mbar_init(smem_u32(&sh.empty[i]), 1);
    }
    for (int i = 0; i < NA; ++i) mbar_init(smem_u32(&sh.ready[i]), 4 * CG);
    for (int i = 0; i < F::kAcc; ++i) {
      mbar_init(smem_u32(&sh.acc_full[i]), 1);
      mbar_init(smem_u32(&sh.acc_empty[i]), F::kEpi * CG);
    }
    mbar_init(smem_u32(&sh.drain), 1);
    for (int i = 0; i < kSegs; ++i) {
      mbar_init(smem_u32(&sh.seg_full[i]), 1);
      // copies, MMAs (one CTA of a pair), conversions, epilogue
      mbar_init(smem_u32(&sh.seg_empty[i]), 2 + (leader ? 1 : 0) + F::kConv + F::kEpi);
    }
    fence_mbar_init();
    sh.abort = 0;
    tma_prefetch_desc(&map_x);
    if (kBatch && p.L > 0 && !p.by_row) tma_prefetch_desc(&map_h);
  }
  if (warp == 1) {
    if constexpr (PAIR) {
      tmem_alloc_pair(smem_u32(&sh.tmem), kTmemCols);
      tmem_relinquish_pair();
    } else {
      tmem_alloc(smem_u32(&sh.tmem), kTmemCols);
      tmem_relinquish();
    }
  }
  pdl_launch_dependents();
  if (prefix != nullptr) {
    // row tiles before each group, by one warp.  Groups of a sort's offsets are
    // disjoint and have max_tiles at most; of offsets that overlap, the tiles
    // from there on are left out, so that the units' k-blocks fit 32 bits.  (A
    // group has R / TN + 1 at most, R / 192 or some 6,000: 32 of them fit too.)
    pdl_wait();
    if (warp == 0) {
      int before = 0;
      for (int e0 = 0; e0 < p.E; e0 += 32) {
        const int e = e0 + lane;
        int n = 0, start;
        if (e < p.E) n = (group_rows(p, e, start) + p.TN - 1) / p.TN;
        int incl = n;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
          const int v = __shfl_up_sync(0xffffffffu, incl, d);
          if (lane >= d) incl += v;
        }
        if (e < p.E) prefix[e] = min(before + incl - n, p.max_tiles);
        before = min(before + __shfl_sync(0xffffffffu, incl, 31), p.max_tiles);
      }
      if (lane == 0) sh.tiles = before;
    }
  } else if (threadIdx.x == 0) {
    sh.tiles = (p.R + p.TN - 1) / p.TN;
  }
  tc_fence_before();
  __syncthreads();
  if constexpr (PAIR) cluster_sync_all();   // the peer's barriers exist before any use
  tc_fence_after();
  const uint32_t tmem = sh.tmem;
  const uint32_t a_base = tmem + F::kAcc * acc_cols;
  volatile uint32_t* abort_flag = &sh.abort;
  const int tiles = sh.tiles;

  if (warp < kFirstConv) {
    split_registers<F::kControlRegs>();
    if (warp == 0) {
      // ---- weights: one elected lane of a warp that runs in step ---------------
      // (a stage's two copies come from two warps: issuing one takes some 200
      // cycles, and a wide stage lasts 384)
      Feed feed{sh};
      const Seg* sg;
      const int64_t w_rows = static_cast<int64_t>(p.KB) * kTileWBytes;
      const uint32_t wfull0 = smem_u32(&sh.wfull[0]), empty0 = smem_u32(&sh.empty[0]);
      // (the weights of a single group need nothing of the kernel before this
      // one: a packed weight is written at load time)
      Ring ring;
      int it = 0;
      bool ok = true;
      while (ok && (sg = feed.next(abort_flag, p.err)) != nullptr) {
        // (an odd last block of a pair repeats the one before and stores nothing)
        const int nb = min(uniform(sg->nb) * CG + rank, p.NB - 1);
        const int kb1 = uniform(sg->kb1);
        const uint8_t* w = p.w + (static_cast<int64_t>(uniform(sg->e)) * p.NB + nb) * w_rows;
        for (int kb = uniform(sg->kb0); kb < kb1; kb += KD, ++it, ring.advance(S)) {
          const uint32_t bytes = min(KD, kb1 - kb) * kTileWBytes;
          ok = tile_wait_warp(empty0 + ring.slot * 8, ring.phase ^ 1, abort_flag, kErrTileRing,
                              p.err);
          if (!ok) break;
          if (elect_one()) {
            const uint32_t bar = wfull0 + ring.slot * 8;
            mbar_arrive_expect_tx(bar, bytes);
            bulk_load(ring0 + ring.slot * stage_bytes + KD * tok_bytes,
                      w + static_cast<int64_t>(kb) * kTileWBytes, bytes, bar);
          }
          __syncwarp();
        }
        if (!ok) break;
        const int na = kBatch ? uniform(sg->na) : 0;
        if (na > 0) pdl_wait();
        const int32_t* list = p.lists + static_cast<int64_t>(sg->tile) * p.list_stride + 1;
        for (int i = 0; i < na && ok; ++i) {
          const int64_t at = static_cast<int64_t>(uniform(list[i])) * p.NB + nb;
          const uint8_t* lb = p.lora_b + at * p.rank16 * 4096;
          for (int c = 0; c < p.rank16; ++c, ++it, ring.advance(S)) {
            ok = tile_wait_warp(empty0 + ring.slot * 8, ring.phase ^ 1, abort_flag, kErrTileRing,
                                p.err);
            if (!ok) break;
            if (elect_one()) {
              const uint32_t bar = wfull0 + ring.slot * 8;
              mbar_arrive_expect_tx(bar, 4096);
              bulk_load(ring0 + ring.slot * stage_bytes + KD * tok_bytes, lb + c * 4096, 4096, bar);
            }
            __syncwarp();
          }
        }
      }
      if (!ok || *abort_flag)   // copies issued but not waited for still land in this CTA
        for (int i = max(0, it - S); i < it; ++i)
          tile_wait_final(smem_u32(&sh.wfull[i % S]), (i / S) & 1);
    } else if (warp == 2) {
      // ---- tokens: likewise ----------------------------------------------------
      pdl_wait();
      Feed feed{sh};
      const Seg* sg;
      const uint32_t tfull0 = smem_u32(&sh.tfull[0]), empty0 = smem_u32(&sh.empty[0]);
      const uint32_t tfull_lead = PAIR ? map_to_cta(tfull0, 0) : tfull0;
      Ring ring;
      int it = 0;
      bool ok = true;
      while (ok && (sg = feed.next(abort_flag, p.err)) != nullptr) {
        const int kb1 = uniform(sg->kb1);
        const int row0 = uniform(sg->row0) + rank * (((uniform(sg->rows) + 15) & ~15) / CG);
        for (int kb = uniform(sg->kb0); kb < kb1; kb += KD, ++it, ring.advance(S)) {
          ok = tile_wait_warp(empty0 + ring.slot * 8, ring.phase ^ 1, abort_flag, kErrTileRing,
                              p.err);
          if (!ok) break;
          if (elect_one()) {
            const uint32_t st = ring0 + ring.slot * stage_bytes;
            if (leader) mbar_arrive_expect_tx(tfull0 + ring.slot * 8, CG * KD * tok_bytes);
            if constexpr (PAIR)
              tma_load_3d_pair(st, &map_x, tfull_lead + ring.slot * 8, 0, row0, kb);
            else
              tma_load_3d(st, &map_x, tfull0 + ring.slot * 8, 0, row0, kb);
          }
          __syncwarp();
        }
        if (!ok) break;
        // adapters: the tile's h, blocks of 16 ranks in place of k-blocks
        const int na = kBatch ? uniform(sg->na) : 0, tile = uniform(sg->tile);
        const int32_t* list = p.lists + static_cast<int64_t>(tile) * p.list_stride + 1;
        const int h0 = row0 - uniform(sg->row0);
        for (int i = 0; i < na && ok; ++i) {
          const int at = (tile + uniform(list[i])) * p.rank16;
          for (int c = 0; c < p.rank16; ++c, ++it, ring.advance(S)) {
            ok = tile_wait_warp(empty0 + ring.slot * 8, ring.phase ^ 1, abort_flag, kErrTileRing,
                                p.err);
            if (!ok) break;
            if (elect_one()) {
              const uint32_t st = ring0 + ring.slot * stage_bytes;
              if (leader) mbar_arrive_expect_tx(tfull0 + ring.slot * 8, CG * tok_bytes);
              if constexpr (PAIR)
                tma_load_3d_pair(st, &map_h, tfull_lead + ring.slot * 8, 0, h0, at + c);
              else
                tma_load_3d(st, &map_h, tfull0 + ring.slot * 8, 0, h0, at + c);
            }
            __syncwarp();
          }
        }
      }
      if ((!ok || *abort_flag) && leader)
        for (int i = max(0, it - S); i < it; ++i)
          tile_wait_final(smem_u32(&sh.tfull[i % S]), (i / S) & 1);
    } else if (warp == 1) {
      // ---- MMAs: one elected lane of a warp that runs in step ------------------
      if (leader) {
        pdl_wait();
        Feed feed{sh};
        const Seg* sg;
        const uint32_t tfull0 = smem_u32(&sh.tfull[0]), empty0 = smem_u32(&sh.empty[0]);
        const uint32_t ready0 = smem_u32(&sh.ready[0]);
        const uint32_t accf0 = smem_u32(&sh.acc_full[0]), acce0 = smem_u32(&sh.acc_empty[0]);
        const uint32_t d0 = uniform(tmem), a0 = d0 + F::kAcc * acc_cols;
        const uint64_t desc0 = sw128_kmajor_desc(0);
        Ring ring, ac;   // stages, accumulators
        int it = 0;
        bool ok = true;
        const int chunk = uniform(chunk_stages_of<KD, kFloat>(p));
        while (ok && (sg = feed.next(abort_flag, p.err)) != nullptr) {
          const uint32_t n16 = uniform((sg->rows + 15) & ~15);
          const uint32_t idesc = idesc_f16(128 * CG, n16);
          int kb = uniform(sg->kb0);
          const int kb1 = uniform(sg->kb1);
          const int stages = (kb1 - kb + KD - 1) / KD;
          for (int c0 = 0; c0 < stages && ok; c0 += chunk, ac.advance(F::kAcc)) {
            const uint32_t buf = ac.slot;
            ok = tile_wait_warp(acce0 + buf * 8, ac.phase ^ 1, abort_flag, kErrTileAcc, p.err);
            if (!ok) break;
            tc_fence_after();
            const uint32_t d = d0 + buf * acc_cols;
            const int c1 = min(stages, c0 + chunk);
            for (int s = c0; s < c1; ++s, ++it, ring.advance(S), kb += KD) {
              const uint32_t as = it & (NA - 1);
              const uint32_t tfull = tfull0 + ring.slot * 8, ready = ready0 + as * 8;
              const uint32_t rphase = (it >> NAb) & 1;
              const bool here = mbar_try_wait(tfull, ring.phase), done = mbar_try_wait(ready, rphase);
              if (!__all_sync(0xffffffffu, here && done)) {
                ok = tile_wait_warp(tfull, ring.phase, abort_flag, kErrTileRing, p.err) &&
                     tile_wait_warp(ready, rphase, abort_flag, kErrTileOperand, p.err);
                if (!ok) break;
              }
              tc_fence_after();
              const uint32_t st = ring0 + ring.slot * stage_bytes;
              const bool two = kb + 1 < kb1;
              if (elect_one()) {
                const uint64_t b = desc0 + (st >> 4);
                const uint32_t a = a0 + as * KD * 32;
#pragma unroll
                for (int j = 0; j < 4; ++j)
                  umma_f16_ta<CG>(d, a + j * 8, b + j * 2, idesc, s > c0 || j > 0);
                if (two) {
                  const uint64_t b1 = b + (tok_bytes >> 4);
#pragma unroll
                  for (int j = 0; j < 4; ++j)
                    umma_f16_ta<CG>(d, a + 32 + j * 8, b1 + j * 2, idesc, 1);
                }
                umma_commit_all<CG>(empty0 + ring.slot * 8);
                if (s + 1 == c1) umma_commit_all<CG>(accf0 + buf * 8);
              }
              __syncwarp();
            }
          }
          if (!ok) break;
          const int na = kBatch ? uniform(sg->na) : 0;
          if (na > 0) {
            const uint32_t buf = ac.slot;
            ok = tile_wait_warp(acce0 + buf * 8, ac.phase ^ 1, abort_flag, kErrTileAcc, p.err);
            if (!ok) break;
            tc_fence_after();
            const uint32_t d = d0 + buf * acc_cols;
            const uint32_t id32 = idesc_tf32(128 * CG, n16);
            const int total = na * p.rank16;
            for (int i = 0; i < total; ++i, ++it, ring.advance(S)) {
              const uint32_t as = it & (NA - 1);
              ok = tile_wait_warp(tfull0 + ring.slot * 8, ring.phase, abort_flag, kErrTileRing,
                                  p.err) &&
                   tile_wait_warp(ready0 + as * 8, (it >> NAb) & 1, abort_flag, kErrTileOperand,
                                  p.err);
              if (!ok) break;
              tc_fence_after();
              if (elect_one()) {
                const uint64_t b = desc0 + ((ring0 + ring.slot * stage_bytes) >> 4);
                const uint32_t a = a0 + as * KD * 32;
#pragma unroll
                for (int j = 0; j < 4; ++j)   // h's leading terms, then its trailing ones
                  umma_tf32_ta<CG>(d, a + (j & 1) * 8, b + j * 2, id32, i > 0 || j > 0);
                umma_commit_all<CG>(empty0 + ring.slot * 8);
                if (i + 1 == total) umma_commit_all<CG>(accf0 + buf * 8);
              }
              __syncwarp();
            }
            ac.advance(F::kAcc);
          }
        }
        if (!ok || *abort_flag) {
          if (elect_one()) {
            umma_commit_own<CG>(smem_u32(&sh.drain));
            tile_wait_final(smem_u32(&sh.drain), 0);
          }
          __syncwarp();
        }
      }
    } else {
      // ---- schedule: the parts of this CTA's units, described for the others ---
      if (kBatch && p.L > 0 && !p.by_row) pdl_wait();   // the tiles' adapters
      Walk<CG> walk(p, prefix, tiles, !kBatch);
      Ring ring;
      bool more = true;
      while (more) {
        Seg sg = {};
        more = walk.next(sg);
        if (kBatch && more) sg.na = adapters_of(p, sg);
        if (!tile_wait_warp(smem_u32(&sh.seg_empty[ring.slot]), ring.phase ^ 1, abort_flag,
                            kErrTileRing, p.err))
          break;
        if (lane == 0) {
          sh.seg[ring.slot] = sg;
          mbar_arrive(smem_u32(&sh.seg_full[ring.slot]));
        }
        __syncwarp();
        ring.advance(kSegs);
      }
    }
  } else if (warp < F::kFirstEpi) {
    split_registers<F::kConvRegs>();
    // ---- A operand: shared memory -> f16 -> TMEM ---------------------------
    const int group = (warp - kFirstConv) >> 2;       // groups take stages in turn
    const int row = (warp & 3) * 32 + lane;           // a warp reaches the lanes of its quarter
    const uint32_t a_lane = a_base + (static_cast<uint32_t>(warp & 3) << 21);
    const __half2 minus = __halves2half2(__ushort_as_half(0x6480), __ushort_as_half(0x6480));
    const uint32_t ready0 = PAIR ? map_to_cta(smem_u32(&sh.ready[0]), 0) : smem_u32(&sh.ready[0]);
    Feed feed{sh};
    const Seg* sg;
    Ring ring, used;   // this stage; the one whose A operand lay where this one's goes
    int it = 0;
    bool ok = true;
    const auto place_free = [&]() {
      return it < NA || tile_wait(smem_u32(&sh.empty[used.slot]), used.phase, abort_flag,
                                  kErrTileOperand, p.err);
    };
    const auto advance = [&]() {
      ring.advance(S);
      if (it >= NA) used.advance(S);
      ++it;
    };
    const auto announce = [&](int as) {
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        if constexpr (PAIR) mbar_arrive_cluster(ready0 + as * 8);
        else mbar_arrive(ready0 + as * 8);
      }
    };
    const auto convert = [&](const uint4 (&v)[4], uint32_t (&r)[32]) {
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const uint32_t q[4] = {v[c].x, v[c].y, v[c].z, v[c].w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          r[c * 8 + j * 2] = biased_to_f16x2(q[j], 0x4140, minus);
          r[c * 8 + j * 2 + 1] = biased_to_f16x2(q[j], 0x4342, minus);
        }
      }
    };
    while (ok && (sg = feed.next(abort_flag, p.err)) != nullptr) {
      for (int kb = sg->kb0; kb < sg->kb1; kb += KD, advance()) {
        if (F::kGroups == 2 && (it & 1) != group) continue;
        const int as = it & (NA - 1);
        const auto landed = [&]() {
          return tile_wait(smem_u32(&sh.wfull[ring.slot]), ring.phase, abort_flag, kErrTileRing,
                           p.err);
        };
        // Two groups: the place first.  It is free once the MMAs of the stage NA
        // back are done, so the slot's last weights, S >= NA stages back, have
        // landed, and the parity below cannot be that of the round before them
        // (which a group that leaves every other stage to its partner has not
        // seen).  One group has seen all weights land, and waits for the place
        // once it has the first ones converted.
        ok = (F::kGroups == 1 || place_free()) && landed();
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        const uint32_t w = ring0 + ring.slot * stage_bytes + KD * tok_bytes + row * 16;
        const bool two = kb + 1 < sg->kb1;
        uint4 v[4], v1[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) v[c] = lds128(w + c * 2048);
        if (two) {
#pragma unroll
          for (int c = 0; c < 4; ++c) v1[c] = lds128(w + kTileWBytes + c * 2048);
        }
        uint32_t r[32];
        convert(v, r);
        if constexpr (F::kGroups == 1) {
          ok = __all_sync(0xffffffffu, place_free());
          if (!ok) break;
        }
        tc_fence_after();
        tmem_st_32cols(a_lane + as * KD * 32, r);
        if (two) {
          convert(v1, r);
          tmem_st_32cols(a_lane + as * KD * 32 + 32, r);
        }
        announce(as);
      }
      if (!ok) break;
      // adapters: B[a]'s blocks of 16 ranks, in tf32
      const int rounds = kBatch ? sg->na * p.rank16 : 0;
      for (int round = 0; round < rounds; ++round, advance()) {
        if (F::kGroups == 2 && (it & 1) != group) continue;
        const int as = it & (NA - 1);
        ok = place_free() && tile_wait(smem_u32(&sh.wfull[ring.slot]), ring.phase, abort_flag,
                                       kErrTileRing, p.err);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        tc_fence_after();
        const uint32_t st = ring0 + ring.slot * stage_bytes;
        uint32_t r[16];
#pragma unroll
        for (int g = 0; g < 2; ++g) {
          const uint4 v = lds128(st + KD * tok_bytes + g * 2048 + row * 16);
          const uint32_t q[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            if (p.lora_f16) {
              const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&q[j]));
              r[g * 8 + j * 2] = __float_as_uint(f.x);
              r[g * 8 + j * 2 + 1] = __float_as_uint(f.y);
            } else {
              r[g * 8 + j * 2] = q[j] << 16;
              r[g * 8 + j * 2 + 1] = q[j] & 0xffff0000u;
            }
          }
        }
        tmem_st_16cols(a_lane + as * KD * 32, r);
        announce(as);
      }
      if (!ok) break;
    }
  } else {
    split_registers<F::kEpiRegs>();
    // ---- epilogue ------------------------------------------------------------
    Feed feed{sh};
    const Seg* sg;
    const int ew = warp - F::kFirstEpi;
    const int quarter = warp & 3;
    // columns of this warp: an equal share of the tile's, in steps of 16
    constexpr int kShares = F::kEpi / 4;
    const int cols = (p.TN + 16 * kShares - 1) / (16 * kShares) * 16;
    const int col0 = (ew / 4) * cols;
    const uint32_t lane_addr = tmem + (static_cast<uint32_t>(quarter) << 21) + col0;
    const uint32_t acce0 =
        PAIR ? map_to_cta(smem_u32(&sh.acc_empty[0]), 0) : smem_u32(&sh.acc_empty[0]);
    const auto release = [&](int buf) {
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        if constexpr (PAIR) mbar_arrive_cluster(acce0 + buf * 8);
        else mbar_arrive(acce0 + buf * 8);
      }
    };
    const int chunk = chunk_stages_of<KD, kFloat>(p);
    const int me = blockIdx.x / CG;
    // the gated gradient: this warp's columns of dh, behind the ring
    auto* my_dh = reinterpret_cast<uint16_t*>(dyn + (ring0 - smem_u32(dyn)) +
                                              static_cast<size_t>(S) * stage_bytes) +
                  ew * (kCols * 16);
    // a CTA's parts: [head of its run, tail, adapter term][kPart]; a warp's
    // words in it as [16 columns][4][lane][4]
    const auto part_at = [&](int cluster, int which) {
      return p.parts + (static_cast<int64_t>(cluster * CG + rank) * 3 + which) * F::kPart +
             ew * (kCols * 32) + lane * 4;
    };
    // The adapters' lines of a part's channels on their way to L2 before they
    // are used: eight lanes a row, 4 lines of 128 bytes to each 8 ranks
    const auto fetch_adapters = [&](const Seg* part, int mine, int nb) {
      for (int j = 0; j < mine; j += 4) {
        const int a = p.ids[part->row0 + min(col0 + j + (lane >> 3), part->rows - 1)];
        if (a >= 0 && a < p.L)
          for (int c = 0; c < p.rank16; ++c)
            prefetch_l2(
                p.lora_b +
                ((static_cast<int64_t>(a) * p.NB + min(nb, p.NB - 1)) * p.rank16 + c) * 4096 +
                ((lane >> 2) & 1) * 2048 + quarter * 512 + (lane & 3) * 128);
      }
    };
    Ring ac;   // accumulators
    bool ok = true, first_seg = true;
    while (ok && (sg = feed.next(abort_flag, p.err)) != nullptr) {
      const int mine = max(0, min(cols, sg->rows - col0));    // columns with a row behind them
      const int stages = (sg->kb1 - sg->kb0 + KD - 1) / KD;
      const int nb = sg->nb * CG + rank;
      if (first_seg) {
        // for the first part even before the kernel before this one is done,
        // where the ids are the caller's; sorted ones are that kernel's, and read
        // now they would lie in L1 as they were before it
        if (!PAIR && kBatch && p.by_row && p.out_rows == nullptr && sg->kb1 == p.KB)
          fetch_adapters(sg, mine, nb);
        pdl_wait();
      }
      TokenScales<FORM> scales;
      if constexpr (!kBatch) scales.load(p, *sg, nb, quarter, col0, mine);
      if constexpr (FORM == kFormGatedGrad) {
        // This part's dh on its way to shared memory while the MMAs run: loads
        // from the epilogue wait behind their tokens and weights (1024 rows x
        // 11008 x 4096: 170 us four at a time, 137 eight).
        __syncwarp();   // the part before has been read
        const int64_t n0 = static_cast<int64_t>(nb) * 64 + quarter * 16 + (lane & 1) * 8;
        const auto* dh = static_cast<const uint16_t*>(p.dh) +
                         static_cast<int64_t>(sg->row0 + col0) * p.N + n0;
        const bool whole = p.N % 8 == 0 && reinterpret_cast<uintptr_t>(p.dh) % 16 == 0;
        for (int j = lane >> 1; j < mine; j += 16) {
          uint16_t* to = my_dh + j * 16 + (lane & 1) * 8;
          const uint16_t* from = dh + static_cast<int64_t>(j) * p.N;
          if (whole) {
            if (n0 < p.N) cp_async16(smem_u32(to), from);
          } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
              if (n0 + i < p.N) to[i] = from[i];
          }
        }
        cp_async_commit();
      }
      // Few rows an adapter: each row's own dot products, put into TMEM columns
      // of their own while the unit's MMAs run
      const bool by_row = !PAIR && kBatch && p.by_row && sg->kb1 == p.KB;
      if (by_row) {
        if (!first_seg || p.out_rows != nullptr) fetch_adapters(sg, mine, nb);
        for (int j = 0; j < mine; j += 8) {
          // (rows past the tile's end repeat its last)
          const int my_s = sg->row0 + min(col0 + j + (lane & 7), sg->rows - 1);
          float d[8];
          row_deltas(p, min(nb, p.NB - 1), quarter * 32 + lane, p.ids[my_s], my_s,
                     sh.corner[ew], d);
          tmem_st_8cols(lane_addr + F::kAcc * acc_cols + NA * KD * 32 + j, d);
        }
        tmem_st_wait();
      }
      int32_t acc[kCols];
#pragma unroll
      for (int j = 0; j < kCols; ++j) acc[j] = 0;
      for (int c0 = 0; c0 < stages; c0 += chunk, ac.advance(F::kAcc)) {
        const int buf = ac.slot;
        ok = __all_sync(0xffffffffu,
                        tile_wait(smem_u32(&sh.acc_full[buf]), ac.phase, abort_flag,
                                  kErrTileAcc, p.err));
        if (!ok) break;
        tc_fence_after();
#pragma unroll
        for (int b = 0; b < kCols / 8; ++b)
          if (b * 8 < mine) {
            uint32_t r[8];
            tmem_ld_8cols(lane_addr + buf * acc_cols + b * 8, r);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              if constexpr (kFloat) acc[b * 8 + j] = static_cast<int32_t>(r[j]);   // one chunk
              else acc[b * 8 + j] += __float2int_rn(__uint_as_float(r[j]));
            }
          }
        release(buf);
      }
      if (!ok) break;
      // the MMAs' adapter term stays in its accumulator until it is used
      const bool by_mma = kBatch && sg->na > 0;
      const int dbuf = ac.slot;
      if (by_mma) {
        ok = __all_sync(0xffffffffu,
                        tile_wait(smem_u32(&sh.acc_full[dbuf]), ac.phase, abort_flag,
                                  kErrTileAcc, p.err));
        if (!ok) break;
        tc_fence_after();
        ac.advance(F::kAcc);
      }
      const bool has_d = by_row || by_mma;
      const uint32_t d_addr =
          lane_addr + (by_row ? F::kAcc * acc_cols + NA * KD * 32 : dbuf * acc_cols);
      // Loops over parts, which a CTA runs once or twice, take 16 columns a
      // round and stay rolled (code that runs once costs more to fetch than to
      // execute): the registers move up by 16 instead.
      const auto rotate = [&]() {
        if constexpr (kCols > 16) {
          int32_t t[16];
#pragma unroll
          for (int j = 0; j < 16; ++j) t[j] = acc[j];
#pragma unroll
          for (int j = 0; j < kCols - 16; ++j) acc[j] = acc[j + 16];
#pragma unroll
          for (int j = 0; j < 16; ++j) acc[kCols - 16 + j] = t[j];
        }
      };
      const bool parted = sg->kb0 != 0 || sg->kb1 != p.KB;
      const int first = sg->first, end = sg->end;
      bool last = true;
      if (parted) {
        // this run holds part of the unit: leave it, and go on only as the last
        int32_t* part = part_at(me, me == first ? 1 : 0);
        int32_t* dpart = part_at(me, 2);
#pragma unroll 1
        for (int b = 0; b < kCols / 16; ++b) {
          if (b * 16 < mine) {
#pragma unroll
            for (int q = 0; q < 4; ++q)
              *reinterpret_cast<int4*>(part + (b * 4 + q) * 128) =
                  make_int4(acc[q * 4], acc[q * 4 + 1], acc[q * 4 + 2], acc[q * 4 + 3]);
            if (has_d) {
#pragma unroll
              for (int half = 0; half < 2; ++half) {
                uint32_t r[8];
                tmem_ld_8cols(d_addr + b * 16 + half * 8, r);
#pragma unroll
                for (int q = 0; q < 2; ++q)
                  *reinterpret_cast<uint4*>(dpart + (b * 4 + half * 2 + q) * 128) =
                      make_uint4(r[q * 4], r[q * 4 + 1], r[q * 4 + 2], r[q * 4 + 3]);
              }
            }
          }
          rotate();
        }
        // release this warp's part, acquire the others'
        __syncwarp();
        int before = 0;
        if (lane == 0)
          before = atomic_add_acq_rel(p.counts + (first * CG + rank) * kTileEpiWarps + ew, 1);
        before = __shfl_sync(0xffffffffu, before, 0);
        __syncwarp();   // lane 0's acquire holds for the others' reads (a shuffle orders none)
        last = before == end - first;
        // (f32 parts are added in their order, whichever CTA does it: its own
        // too is taken from where it left it)
        if constexpr (kFloat) {
          if (last)
#pragma unroll
            for (int j = 0; j < kCols; ++j) acc[j] = 0;
        }
        if (last) {
#pragma unroll 1
          for (int b = 0; b < kCols / 16; ++b) {
            if (b * 16 < mine) {
              // the narrow form has registers for three parts' loads at once
              // (this CTA's own place, and places past the last, are zeros)
              constexpr int kAtOnce = 3;
              if constexpr (PAIR) {
                for (int c = first; c <= end; ++c) {
                  if (!kFloat && c == me) continue;
                  const int32_t* other = part_at(c, c == first ? 1 : 0);
#pragma unroll
                  for (int q = 0; q < 4; ++q) {
                    const int4 v = __ldcg(reinterpret_cast<const int4*>(other + (b * 4 + q) * 128));
                    add_part<kFloat>(acc[q * 4], v.x);
                    add_part<kFloat>(acc[q * 4 + 1], v.y);
                    add_part<kFloat>(acc[q * 4 + 2], v.z);
                    add_part<kFloat>(acc[q * 4 + 3], v.w);
                  }
                }
              } else {
                for (int c0 = first; c0 <= end; c0 += kAtOnce) {
                  int4 v[kAtOnce][4];
#pragma unroll
                  for (int k = 0; k < kAtOnce; ++k) {
                    const int c = c0 + k;
                    const bool use = c <= end && (kFloat || c != me);
                    const int32_t* other = part_at(use ? c : me, c == first ? 1 : 0);
#pragma unroll
                    for (int q = 0; q < 4; ++q)
                      v[k][q] =
                          use ? __ldcg(reinterpret_cast<const int4*>(other + (b * 4 + q) * 128))
                              : make_int4(0, 0, 0, 0);
                  }
#pragma unroll
                  for (int k = 0; k < kAtOnce; ++k)
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                      add_part<kFloat>(acc[q * 4], v[k][q].x);
                      add_part<kFloat>(acc[q * 4 + 1], v[k][q].y);
                      add_part<kFloat>(acc[q * 4 + 2], v[k][q].z);
                      add_part<kFloat>(acc[q * 4 + 3], v[k][q].w);
                    }
                }
              }
            }
            rotate();
          }
        }
      }
      if constexpr (!kBatch) {
        if constexpr (FORM == kFormGatedGrad) {
          cp_async_wait<0>();
          __syncwarp();
        }
        if (last && mine > 0)
          token_epilogue<OUT, kCols, FORM>(p, *sg, acc, scales, nb, quarter, col0, mine, my_dh);
        first_seg = false;
        continue;
      }
      const int n = nb * 128 + quarter * 32 + lane;
      const bool in = n < p.N;
      if (last) {
        // In place from here on: registers beyond the sums are few, and what
        // spills finds no L1 beside this much shared memory.
        const int64_t en = static_cast<int64_t>(sg->e) * p.N + n;
        const float ws = in ? __ldg(p.ws + en) : 0.0f;
        const float bias = in && p.bias != nullptr ? __ldg(p.bias + en) : 0.0f;
        // (the narrow form skips columns without rows; in the wide one the
        // branches cost registers that spill)
#pragma unroll
        for (int b = 0; b < kCols; b += 16)
          if (PAIR || b < mine)
#pragma unroll
            for (int j = b; j < b + 16; ++j)
              acc[j] = __float_as_int(dequant(acc[j], ws, bias, p.rq));
        // the unit's adapter term: in this CTA's TMEM, or left by the CTA
        // that ran the unit's end
        const bool other_d =
            !has_d && p.L > 0 &&
            (p.by_row || p.lists[static_cast<int64_t>(sg->tile) * p.list_stride] > 0);
        if (has_d) {
#pragma unroll
          for (int b = 0; b < kCols / 8; ++b)
            if (b * 8 < mine) {
              uint32_t r[8];
              tmem_ld_8cols(d_addr + b * 8, r);
#pragma unroll
              for (int j = 0; j < 8; ++j)
                acc[b * 8 + j] = __float_as_int(
                    __fadd_rn(__int_as_float(acc[b * 8 + j]), __uint_as_float(r[j])));
            }
        } else if (other_d) {
          const int32_t* dpart = part_at(end, 2);
#pragma unroll 1
          for (int b = 0; b < kCols / 16; ++b) {
            if (b * 16 < mine) {
#pragma unroll
              for (int q = 0; q < 4; ++q) {
                const int4 v = __ldcg(reinterpret_cast<const int4*>(dpart + (b * 4 + q) * 128));
                const int32_t r[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int j = 0; j < 4; ++j)
                  acc[q * 4 + j] = __float_as_int(
                      __fadd_rn(__int_as_float(acc[q * 4 + j]), __int_as_float(r[j])));
              }
            }
            rotate();
          }
        }
      }
      if (by_mma) release(dbuf);   // before the stores, which take longest
      if (last && mine > 0) {
        using T = typename OutType<OUT>::type;
        if (p.out_rows == nullptr) {
          // one address for the tile and 32-bit distances from it (a tile's
          // rows span less than 4 GB: N <= 2^24)
          char* base = static_cast<char*>(p.out) +
                       static_cast<int64_t>(sg->row0 + col0) * p.N * sizeof(T);
          const uint32_t step = static_cast<uint32_t>(p.N) * sizeof(T);
          uint32_t off = static_cast<uint32_t>(n) * sizeof(T);
          if (mine == kCols && in) {
#pragma unroll
            for (int j = 0; j < kCols; ++j, off += step)
              *reinterpret_cast<T*>(base + off) = finish<OUT>(__int_as_float(acc[j]), p);
          } else {
            const int rows = in ? mine : 0;
#pragma unroll
            for (int b = 0; b < kCols; b += 8)
              if (PAIR || b < mine)
#pragma unroll
                for (int j = b; j < b + 8; ++j, off += step)
                  if (j < rows)
                    *reinterpret_cast<T*>(base + off) = finish<OUT>(__int_as_float(acc[j]), p);
          }
        } else {
          // a lane looks up one or two columns' rows for all of them
          T* to = static_cast<T*>(p.out) + n;
          const int32_t* map = p.out_rows + sg->row0 + col0;
          const int m0 = map[min(lane, mine - 1)];
          const int m1 = kCols > 32 ? map[min(lane + 32, mine - 1)] : 0;
#pragma unroll
          for (int j = 0; j < kCols; ++j) {
            const int64_t row = __shfl_sync(0xffffffffu, j < 32 ? m0 : m1, j & 31);
            if (in && j < mine) to[row * p.N] = finish<OUT>(__int_as_float(acc[j]), p);
          }
        }
      }
      first_seg = false;
    }
    if constexpr (FORM == kFormGatedGrad) cp_async_wait<0>();   // (where the loop was left early)
    if (first_seg) pdl_wait();
    // rows of dropped slots hold zeros
    if (prefix != nullptr) {
      const int64_t step = static_cast<int64_t>(gridDim.x) * F::kEpi * 32;
      const int64_t total = static_cast<int64_t>(p.R) * p.N;
      for (int64_t i = group_end(p, p.E) * static_cast<int64_t>(p.N) +
                       static_cast<int64_t>(blockIdx.x) * F::kEpi * 32 + ew * 32 + lane;
           i < total; i += step) {
        if constexpr (OUT == Q8_I8)
          static_cast<int8_t*>(p.out)[i] = static_cast<int8_t>(p.rq.ozp_i);
        else if constexpr (OUT == Q8_F32) static_cast<float*>(p.out)[i] = 0.0f;
        else static_cast<uint16_t*>(p.out)[i] = 0;
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  // neither CTA of a pair leaves while the leader's MMAs may still read the
  // peer's memories or arrive at its barriers
  if constexpr (PAIR) cluster_sync_all();
  tc_fence_after();
  if (warp == 1) {
    if constexpr (PAIR) tmem_dealloc_pair(tmem, kTmemCols);
    else tmem_dealloc(tmem, kTmemCols);
  }
}

template <int OUT, bool PAIR, TileForm FORM>
cudaError_t launch_one(const CUtensorMap& map, const CUtensorMap& map_h, const TileParams& p,
                       size_t smem, cudaStream_t s) {
  constexpr int CG = Form<PAIR>::CG;
  auto kernel = tile_gemm_kernel<OUT, PAIR, FORM>;
  static DeviceOnce once;
  static int fit[64];   // by device; written once, under the lock that every reader takes first
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  int pairs = 0;
  e = once.run([&] {
    cudaFuncAttributes attributes;
    cudaError_t set = cudaFuncGetAttributes(&attributes, kernel);
    if (set != cudaSuccess) return set;
    if (attributes.numRegs < Form<PAIR>::kRegs) return cudaErrorInvalidConfiguration;
    set = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kTileSmem);
    if (!PAIR || set != cudaSuccess) return set;
    // pairs that fit the GPU at once (both CTAs of one share a GPC)
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = p.grid / CG * CG;
    cfg.blockDim = kTileThreads;
    cfg.dynamicSmemBytes = kTileSmem;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = CG;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaOccupancyMaxActiveClusters(&pairs, kernel, &cfg) != cudaSuccess || pairs <= 0) {
      cudaGetLastError();
      pairs = p.grid / CG;
    }
    if (dev >= 0 && dev < 64) fit[dev] = pairs;
    return cudaSuccess;
  });
  if (e != cudaSuccess) return e;
  if constexpr (PAIR) {
    if (pairs == 0) pairs = fit[dev];
    const int grid = std::max(1, std::min(pairs, p.grid / CG)) * CG;
    return launch_pdl_cluster(kernel, grid, kTileThreads, smem, CG, s, map, map_h, p);
  } else {
    return launch_pdl(kernel, p.grid, kTileThreads, smem, s, map, map_h, p);
  }
}

template <bool PAIR, TileForm FORM>
cudaError_t launch_form(TileParams p, const void* operand, q8_dtype out_dtype, cudaStream_t s) {
  using F = Form<PAIR>;
  CUtensorMap map;
  const uint64_t dims[3] = {64, static_cast<uint64_t>(p.R), static_cast<uint64_t>(p.KB)};
  const uint64_t str[2] = {128, static_cast<uint64_t>(p.R) * 128};
  const uint32_t box[3] = {64, static_cast<uint32_t>(p.TN / F::CG), F::KD};
  // (16-bit elements; the map's element type only matters for reductions)
  if (!encode_bf16_tmap(&map, operand, 3, dims, str, box)) return cudaErrorInvalidValue;
  CUtensorMap map_h = map;
  if (p.L > 0 && !p.by_row) {
    // h in rows of 16 leading and 16 trailing f32 terms
    const int64_t blocks =
        (static_cast<int64_t>((p.R + p.TN - 1) / p.TN) + p.L) * p.rank16;
    const uint64_t dims_h[3] = {64, static_cast<uint64_t>(p.TN), static_cast<uint64_t>(blocks)};
    const uint64_t str_h[2] = {128, static_cast<uint64_t>(p.TN) * 128};
    const uint32_t box_h[3] = {64, static_cast<uint32_t>(p.TN / F::CG), 1};
    if (!encode_bf16_tmap(&map_h, p.h, 3, dims_h, str_h, box_h)) return cudaErrorInvalidValue;
  }
  const size_t stage = static_cast<size_t>(F::KD) * (p.TN / F::CG * 128 + kTileWBytes);
  // behind the ring: tiles before each group, or the epilogue's dh
  const size_t table = FORM == kFormGatedGrad  ? static_cast<size_t>(F::kEpi) * F::kCols * 32
                       : p.offsets != nullptr ? (static_cast<size_t>(p.E) + 1) * 4
                                              : 0;
  p.stages = static_cast<int>(std::min<size_t>(F::kRing, (kTileSmem - 1024 - table) / stage));
  const size_t smem = 1024 + table + static_cast<size_t>(p.stages) * stage;
  constexpr bool kSixteen = FORM == kFormGatedGrad || FORM == kFormGrad;
  switch (out_dtype) {
    case Q8_F16: return launch_one<Q8_F16, PAIR, FORM>(map, map_h, p, smem, s);
    case Q8_BF16: return launch_one<Q8_BF16, PAIR, FORM>(map, map_h, p, smem, s);
    case Q8_F32:
      if constexpr (!kSixteen) return launch_one<Q8_F32, PAIR, FORM>(map, map_h, p, smem, s);
      break;
    case Q8_I8:
      if constexpr (FORM == kFormBatch) return launch_one<Q8_I8, PAIR, FORM>(map, map_h, p, smem, s);
      break;
  }
  return cudaErrorInvalidValue;
}

// By the tiles' height: narrow up to 64 rows, else wide.
template <TileForm FORM>
cudaError_t launch_tiles(TileParams p, const void* operand, q8_dtype out_dtype, cudaStream_t s) {
  p.err = device_error_word();
  if (p.err == nullptr) return cudaErrorUnknown;
  return p.TN > Form<false>::kMaxRows ? launch_form<true, FORM>(p, operand, out_dtype, s)
                                      : launch_form<false, FORM>(p, operand, out_dtype, s);
}

}  // namespace

}  // namespace q8
