// tile_plan.h -- host side of the int8-weight contraction (tile_gemm_kernel.cuh):
// sizes it takes, tile height, grid and workspace.  Shared by the entry points.
#pragma once

#include <algorithm>
#include <cstdint>

#include "api_common.h"
#include "rows_internal.h"

namespace q8api {

inline bool aligned(const void* p, int64_t bytes) {
  return reinterpret_cast<uintptr_t>(p) % static_cast<uintptr_t>(bytes) == 0;
}

inline size_t tile_weight_bytes(int64_t E, int64_t N, int64_t K) {
  return static_cast<size_t>(E) * ((N + 127) / 128) * ((K + 63) / 64) * 8192;
}

inline bool tile_sizes_ok(int64_t E, int64_t N, int64_t K) {
  return E >= 1 && E <= q8::kMaxExperts && N >= 1 && K >= 1 && N <= (1 << 24) &&
         K <= INT32_MAX / 2 && mul_ok(N, K) && mul_ok(E, N * K) && E * N * K <= INT64_MAX / 64;
}

// Tile height and grid of a problem of R rows in E groups.
struct TilePlan {
  int TN, grid;
  size_t operand, parts, counts, total;
};

inline TilePlan plan_tiles(int64_t R, int64_t K, int64_t E, int64_t max_rows = q8::kMaxTileRows) {
  TilePlan t{};
  // tiles hold twice the average group, so that few groups need a second one
  // (which reads the weights again)
  const int64_t groups = std::min(E, R), avg = (R + groups - 1) / groups;
  const int64_t want = E == 1 ? avg : 2 * avg;
  t.TN = static_cast<int>(std::min<int64_t>(max_rows, q8::round_up(want, 16)));
  t.grid = q8::device_sm_count();
  t.operand = q8::align_ws(static_cast<size_t>(R) * q8::round_up(K, q8::kTileK) * 2);
  t.parts = q8::align_ws(static_cast<size_t>(t.grid) * 3 * q8::kTilePartWords * 4);
  t.counts = q8::align_ws(static_cast<size_t>(t.grid) * q8::kTileEpiWarps * 4);
  t.total = t.operand + t.parts + t.counts;
  return t;
}

// The tile height of one group of R rows, N packed rows and K inputs: the one
// whose slowest CTA (or pair) is done first, by the split that the kernel's Walk
// makes of it.  Low tiles make more units, which a few rows need to fill the GPU
// without cutting units (a join costs 3 us and more); high ones read the weights
// less often, and stay where a lower one gains less than 3%.  The constants (ns:
// the launches, a k-block, a unit's epilogue, a join and its parts) were fitted to
// 195 problems of 20 to 2000 rows, all forms, to 7%; the choice is then within
// 1.7% of the best height (16% at worst), where full tiles take 18% longer (2.4
// times at worst: 70 rows, 5000 inputs, 512 outputs 22.7 us against 12.0).
inline int64_t tile_time(int64_t R, int64_t N, int64_t K, int TN, int grid, int min_run) {
  const bool wide = TN > q8::kMaxNarrowRows;
  const int64_t ctas = std::max(1, wide ? grid / 2 : grid), KB = (K + 63) / 64;
  const int64_t blocks = (N + 127) / 128, tiles = (R + TN - 1) / TN;
  const int64_t rows = ((R + tiles - 1) / tiles + 15) / 16 * 16;
  const int64_t units = tiles * (wide ? (blocks + 1) / 2 : blocks), full = units / ctas;
  const int64_t behind = units - full * ctas;
  const int64_t waves =
      behind == 0 || behind >= ctas / 4 ? full : std::max<int64_t>(full - 1, 0);
  const int64_t rest = units - waves * ctas, total = rest * KB;
  int64_t line = 0, ends = 0, parts = 0;   // k-blocks, units and parts to join
  if (rest > 0) {
    const bool few = 2 * rest <= ctas;
    const int64_t whole = (rest + ctas - 1) / ctas * KB;
    int64_t q = std::max<int64_t>(min_run, (total - 1) / ctas + 1);
    if (whole <= q + (wide ? q8::kJoinWide : q8::kJoinNarrow)) q = whole;
    ends = std::max<int64_t>(1, (q + KB - 1) / KB);
    if (few && q < KB) {
      const int64_t share = std::max<int64_t>(1, std::min(ctas / rest, KB / std::max(1, min_run)));
      line = (KB + share - 1) / share;
      ends = 1;
      parts = share > 1 ? share : 0;
    } else {
      line = std::min(q, total);
      if (q % KB != 0 && q < total) parts = (KB + q - 1) / q + 1;
    }
  }
  const int64_t kbs = waves * KB + line, epilogues = waves + ends;
  if (wide)
    return 5900 + kbs * (1380 + 3 * rows) / 10 + epilogues * std::max<int64_t>(0, 21 * rows - 500) +
           (parts > 0 ? 4900 + parts * rows * 7 : 0);
  return 4900 + kbs * (1190 + 4 * rows) / 10 + epilogues * (270 + 16 * rows) +
         (parts > 0 ? 3200 + parts * rows * 6 : 0);
}

// Row tiles that R rows in E groups need at most.
inline int64_t max_tiles(int64_t R, int64_t E, const TilePlan& t) { return R / t.TN + std::min(E, R); }

// The k-blocks of all units are numbered in 32 bits.
inline bool units_ok(int64_t R, int64_t E, int64_t N, int64_t K, const TilePlan& t) {
  const int64_t tiles = max_tiles(R, E, t), blocks = (N + 127) / 128, kbs = (K + 63) / 64;
  return mul_ok(blocks, kbs) && mul_ok(tiles, blocks * kbs) && tiles * blocks * kbs <= INT32_MAX;
}

// A plan of one group, by tile_time (its workspace is plan_tiles's: heights do not
// change it).  A program asks for the same few sizes again and again, and twelve
// heights take the host 1 us: a thread remembers sixteen answers.
inline TilePlan plan_group(int64_t R, int64_t N, int64_t K, int min_run) {
  TilePlan t = plan_tiles(R, K, 1);
  struct Known {
    int64_t R, N, K;
    int grid, min_run, TN;
  };
  static thread_local Known all[16] = {};
  Known& known = all[(R * 31 + N * 7 + K) & 15];
  if (known.R == R && known.N == N && known.K == K && known.grid == t.grid &&
      known.min_run == min_run) {
    t.TN = known.TN;
    return t;
  }
  const int full = t.TN;   // as high as there are rows for
  int64_t best = INT64_MAX;
  TilePlan c = t;
  for (int height = full; height > 0; height -= 16) {
    c.TN = height;
    if (!units_ok(R, 1, N, K, c)) continue;
    const int64_t time = tile_time(R, N, K, height, t.grid, min_run);
    if (best == INT64_MAX || time < best / 100 * 97) {
      best = time;
      t.TN = height;
    }
  }
  known = {R, N, K, t.grid, min_run, t.TN};
  return t;
}

}  // namespace q8api
