// token_internal.h -- host-side declarations of the operators for rows with a
// scale for each token (token_kernels.cu): quantizing them and back, and what
// the contraction (rows_internal.h) reads beside a packed weight.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

#include "q8ta.h"
#include "rows_internal.h"

namespace q8 {

// Rows [M, K] of float type to int8, each with its own scale; where asked,
// also the contraction's operand (f16, K-blocked, see launch_tile_operand) and
// `counts` zeroed.
struct QuantizeJob {
  const void* x;
  int64_t M, K;
  int8_t* q;         // or null
  float* scales;     // [M]
  uint16_t* operand; // [KB][M][64], or null
  int KB;
  int32_t* counts;
  int count_words;
};
cudaError_t launch_quantize_token(const QuantizeJob& job, q8_dtype dtype, cudaStream_t s);
cudaError_t launch_dequantize_token(const int8_t* q, const float* scales, int64_t M, int64_t K,
                                    q8_dtype dtype, void* out, cudaStream_t s);

// dst[kb][m][64] = f16(dy[m, n] * ws[n] * rescale[m]), dy as 0 where y is given
// and not above 0, and zeros for N <= n < 64 KB; unscale[m] = 1 / rescale[m];
// `counts` zeroed.
struct GradOperandJob {
  const void *dy, *y;   // [M, N]; y or null
  const float* ws;      // [N]
  int64_t M, N;
  uint16_t* dst;
  float* unscale;       // [M]
  int KB;
  int32_t* counts;
  int count_words;
};
cudaError_t launch_grad_operand(const GradOperandJob& job, q8_dtype dtype, cudaStream_t s);

// What the gated gradient's kernel reads: the int8 rows' operand, each row's
// largest |dh|, the largest scales and biases, `counts` zeroed.
struct GatedGradFrontJob {
  const int8_t* q;      // [M, K]
  const void* dh;       // [M, N]
  const float *ws, *bias;   // [2, N]; bias or null
  int64_t M, N, K;
  uint16_t* operand;    // [KB][M][64]
  int KB;
  float* most_dh;       // [M]
  float* tops;          // [4]: of the gate's and the up projection's ws, and of their biases
  int32_t* counts;
  int count_words;
};
cudaError_t launch_gated_grad_front(const GatedGradFrontJob& job, q8_dtype dtype, cudaStream_t s);

// Products of up to kFewRows short rows in one launch without a workspace
// (token_rows.cu; token_rows_fit says which).
constexpr int kFewRows = 8;
struct TokenRowsJob {
  const void* x;        // [M, K] of x_dtype
  q8_dtype x_dtype;
  int64_t M, K;
  int8_t* q;            // float x: its int8 rows, or null
  float* scales;        // int8 x: read; float x: written, or null
  const uint8_t* w;     // packed
  int64_t N;            // output channels
  const float *ws, *bias;   // [N], or [2, N] of a gated pair
  int act;
  q8_dtype out_dtype;
  void* out;            // [M, N]
  int KB, stride, units, vec;   // set by the launcher
};
// Bytes of an int8 row in shared memory: 64 more than a multiple of 128, so that
// two rows' 64 bytes of one k-block meet no bank twice.
inline int64_t token_rows_stride(int64_t K) { return round_up(round_up(K, 64) - 64, 128) + 64; }
// copied: int8 rows for a product by one weight.
bool token_rows_fit(int64_t M, int64_t K, bool copied);
cudaError_t launch_token_rows(TokenRowsJob job, bool gated, cudaStream_t s);

// A gated weight's two halves [N, K] in tiles: rows 16 of the gate and 16 of
// the up projection in turn (gated_rows), or transposed: K rows of that many
// inputs.
cudaError_t launch_pack_gated(const int8_t* gate, const int8_t* up, int64_t N, int64_t K,
                              bool transposed, uint8_t* dst, cudaStream_t s);

}  // namespace q8
