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

// Row tiles that R rows in E groups need at most.
inline int64_t max_tiles(int64_t R, int64_t E, const TilePlan& t) { return R / t.TN + std::min(E, R); }

// The k-blocks of all units are numbered in 32 bits.
inline bool units_ok(int64_t R, int64_t E, int64_t N, int64_t K, const TilePlan& t) {
  const int64_t tiles = max_tiles(R, E, t), blocks = (N + 127) / 128, kbs = (K + 63) / 64;
  return mul_ok(blocks, kbs) && mul_ok(tiles, blocks * kbs) && tiles * blocks * kbs <= INT32_MAX;
}

}  // namespace q8api
