// row_split.h -- index arithmetic of the kernels for rows of one batch, in
// steps that stay within their types for every size the host lets through.
// Plain C++ on the host; no CUDA header is needed to include it.
#pragma once

#include <cstdint>

#ifdef __CUDACC__
#define Q8_HOST_DEVICE __host__ __device__ __forceinline__
#else
#define Q8_HOST_DEVICE inline
#endif

namespace q8 {

// Items first, first + step, ... of rows of `width` items each, as (row, item):
// two divisions at the start and none after, whatever rows * width is.
struct RowItems {
  int64_t row;
  uint32_t item;
  uint32_t rows_step, items_step, width;
  Q8_HOST_DEVICE RowItems(uint32_t first, uint32_t step, uint32_t width_)
      : row(first / width_), item(first % width_), rows_step(step / width_),
        items_step(step % width_), width(width_) {}
  Q8_HOST_DEVICE void next() {
    row += rows_step;
    item += items_step;
    if (item >= width) {
      item -= width;
      ++row;
    }
  }
};

// part * n / parts, 0 <= part <= parts <= 2^15: where part `part` of n steps cut
// into equal `parts` begins.  No product passes n or parts^2.
Q8_HOST_DEVICE int part_start(int part, int n, int parts) {
  return part * (n / parts) + part * (n % parts) / parts;
}

}  // namespace q8
