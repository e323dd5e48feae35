// token_split.h -- which of a row's items of 8 values a warp's lanes take in the
// quantizer (token_kernels.cu).  Plain C++ on the host; no CUDA header is needed
// to include it.
#pragma once

#include "row_split.h"

namespace q8 {

// OP: the row is also written as the product's operand; VEC: rows are whole items.
// A row that begins t < 8 values into its first item reaches up to item
// (t + K - 1) / 8.  The operand's items begin with the row, so a lane puts one
// together from its own and the next lane's: a warp's last lane then only lends,
// and its item is the next warp's first.
template <bool VEC, bool OP>
struct RowLanes {
  static constexpr int kStoring = !VEC && OP ? 31 : 32;   // of a warp's 32 lanes
  static Q8_HOST_DEVICE int first(int warp, int lane) { return warp * kStoring + lane; }
  static Q8_HOST_DEVICE int step(int warps) { return warps * kStoring; }
  static Q8_HOST_DEVICE bool stores(int lane) { return kStoring == 32 || lane < kStoring; }
  // Items that whole warps go through: all that a row of K values can reach, and
  // the operand's `chunks`.  (Either can be more: K 1983 has 248 chunks, and from
  // t = 2 on an item 248, which 8 warps of 31 lanes that store do not reach.)
  static Q8_HOST_DEVICE int items(int K, int chunks) {
    const int row = (K + (VEC ? 7 : 14)) / 8;
    return OP && chunks > row ? chunks : row;
  }
};

}  // namespace q8
