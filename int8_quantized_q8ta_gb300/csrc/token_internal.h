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

// dst[kb][m][64] = dy[m, n] * ws[n] * *rescale (null: 1) in dy's type, 0 where
// y is given and not above 0, and for N <= n < 64 KB; `counts` zeroed.
struct GradOperandJob {
  const void *dy, *y;   // [M, N]; y or null
  const float *ws, *rescale;
  int64_t M, N;
  uint16_t* dst;
  int KB;
  int32_t* counts;
  int count_words;
};
cudaError_t launch_grad_operand(const GradOperandJob& job, q8_dtype dtype, cudaStream_t s);

// norm[0] = 2^-e and norm[1] = 2^e with e the exponent of the largest |ws|.
cudaError_t launch_channel_norm(const float* ws, int64_t n, float* norm, cudaStream_t s);

// A gated weight's two halves [N, K] in tiles: rows 16 of the gate and 16 of
// the up projection in turn (gated_rows), or transposed: K rows of that many
// inputs.
cudaError_t launch_pack_gated(const int8_t* gate, const int8_t* up, int64_t N, int64_t K,
                              bool transposed, uint8_t* dst, cudaStream_t s);
// word[0] = max(word[0], word[1])
cudaError_t launch_larger_bound(int32_t* word, cudaStream_t s);

}  // namespace q8
