// rows_internal.h -- host-side declarations of the operators for rows of one
// batch that go through different weights: the expert sort and its row moves
// (route_kernels.cu), and the grouped int8 contraction (tile_gemm.cu).
#pragma once

#include <cuda_runtime.h>

#include <cstdint>
#include <mutex>

#include "q8ta.h"
#include "q8ta_internal.h"

namespace q8 {

constexpr int kMaxExperts = 1024;  // the sort's per-warp counts fill shared memory

inline int64_t dtype_bytes(q8_dtype dt) { return dt == Q8_F32 ? 4 : dt == Q8_I8 ? 1 : 2; }

// A one-time set-up per device (kernel attributes).
class DeviceOnce {
 public:
  template <typename F>
  cudaError_t run(F&& f) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return f();
    std::lock_guard<std::mutex> lock(mu_);
    if (done_[dev]) return cudaSuccess;
    e = f();
    done_[dev] = e == cudaSuccess;
    return e;
  }

 private:
  std::mutex mu_;
  bool done_[64] = {false};
};

// launch_pdl with thread-block clusters of `cluster` CTAs along x.
template <typename... KArgs, typename... Args>
inline cudaError_t launch_pdl_cluster(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem,
                                      int cluster, cudaStream_t s, Args&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, static_cast<KArgs>(args)...);
  if (e != cudaSuccess) return e;
  return cudaGetLastError();
}

// ---- expert sort and row moves (route_kernels.cu) -------------------------
// keep_dropped: the dropped slots keep their places at the end of order.
cudaError_t launch_expert_sort(const int32_t* ids, int64_t R, int E, int32_t* order,
                               int32_t* position, int32_t* offsets, cudaStream_t s,
                               bool keep_dropped = false);
cudaError_t launch_expert_gather(const void* x, int64_t T, int k, int64_t row_bytes,
                                 const int32_t* position, const int32_t* offsets, int E, void* xs,
                                 cudaStream_t s);
cudaError_t launch_expert_dispatch(const void* x, int64_t T, int k, int64_t row_bytes,
                                   const int32_t* ids, int E, int32_t* order, int32_t* position,
                                   int32_t* offsets, void* xs, cudaStream_t s);
// y[t] = sum_j w[t,j] * z[position[t,j]]; w null: ones.
cudaError_t launch_expert_spread(const void* z, q8_dtype dt, const float* w, int64_t T, int k,
                                 int64_t H, const int32_t* position, void* y, cudaStream_t s);
cudaError_t launch_expert_combine_bwd(const void* dy, const void* z, q8_dtype dt, const float* w,
                                      int64_t T, int k, int64_t H, const int32_t* position,
                                      const int32_t* offsets, int E, void* dz, float* dw,
                                      cudaStream_t s);

// ---- grouped int8 contraction (tile_gemm.cu, tile_prep.cu) -----------------
constexpr int kMaxTileRows = 192;       // rows of one tile: two accumulators fit TMEM
constexpr int kMaxNarrowRows = 64;   // of the form of one CTA
constexpr int kMaxByRow = 64;           // rows of a tile whose adapter terms go row by row
constexpr int kTileEpiWarps = 12;       // epilogue warps at most
constexpr int kTilePartWords = kMaxTileRows * 128;   // int32 words of one CTA's part of a unit
constexpr int kTileSmem = 218 * 1024;   // beside it some 7 KB of static shared memory
constexpr int kMaxRank = 256;

// Rows of each tile of a group of `count` rows cut into `tiles`: equal
// shares in steps of 16 (at most kMaxTileRows, as tiles >= count / that).
__host__ __device__ inline int tile_rows(int count, int tiles) {
  return ((count + tiles - 1) / tiles + 15) & ~15;
}

// Whole units to each CTA while that lengthens the longest run by no more than
// this many k-blocks over equal runs, which cut units and then join their
// parts (5,000 to 10,000 cycles a join, against 350 a narrow k-block and 400 a
// wide one; a run across two units joins twice).  Measured, whole against cut,
// K 4096: 64 rows x 11008 (27 k-blocks more) 19.9 against 22.9 us, x 28672 (33)
// 31.6 against 34.4, x 8192 (37) 19.0 against 18.7, 8 rows x 22016 (55) 26.8
// against 26.0, x 6144 (43) 16.9 against 15.1; wide, 192 rows x 11008 (27) 27.3
// against 37.2, 100 rows x 4096 (37) 24.9 against 22.3.  With adapters row by
// row a second unit's terms are made once its first is joined, and whole units
// win further: 8 and 64 rows x 22016 25.8 against 28.4 and 44 against 50.
constexpr int kJoinNarrow = 36, kJoinWide = 28, kJoinByRow = 60;

struct TileParams {
  int R, N, NB, KB;         // rows, output channels, blocks of 128 of them, k-blocks of 64
  int E;                    // groups
  const int32_t* offsets;   // [E + 1] group bounds on the device, or null: one group of R rows
  int TN;                   // rows of a tile at most (a multiple of 16)
  int max_tiles;            // row tiles of all groups at most: R / TN + min(E, R)
  int stages;               // ring stages (set by the launcher)
  int grid, min_run;        // CTAs; k-blocks a CTA's run holds at least
  const uint8_t* w;         // packed weights (see launch_pack_tile_weight)
  const int32_t* w_bound;   // largest sum of |w| over 64 inputs
  int a_bound;              // largest |x - zp|
  const float* ws;          // [E, N]
  const float* bias;        // [E, N] or null
  Requant rq;
  float floor_f;            // float outputs below it become 0: 0 for relu, -inf for none
  void* out;
  const int32_t* out_rows;  // output row of each row, or null
  uint32_t* err;
  int32_t* parts;           // [grid][3][words]: parts of units cut by a run's end
  int32_t* counts;          // [grid][kTileEpiWarps], zeroed by the kernel before
  // adapters (L == 0: none)
  int L, rank16, lora_f16;  // adapters, blocks of 16 ranks, f16 (1) or bf16 (0)
  int by_row;               // the term row by row in the epilogue (TN <= kMaxByRow), not by MMAs
  const uint8_t* lora_b;    // packed B (see launch_pack_lora)
  const float* h;           // s_in * scaling * (x - zp) A^T, as by_row wants it (store_h)
  const int32_t* ids;       // [R] adapter of each row
  const int32_t* lists;     // per row tile: adapter count, then the adapters
  int list_stride;
  // rows with a scale for each token (L == 0, offsets null, E == 1)
  const float* row_scale;   // [R]
  int act;                  // Activation of the gated forms
  const void* dh;           // [R, N] the gated output's gradient
  uint16_t* operand_out;    // [2 NB][R][64] the gradient's operand, f16
  int64_t K;                // the gated gradient: inputs of a row, and with
  const float* most_dh;     // [R] its largest |dh| and the largest scales and
  const float* tops;        // [4] biases (see gated_row_power) the powers of two
  float* unscale;           // [R] that its operand is multiplied by; what the
                            // next kernel's sums are multiplied by
};
cudaError_t launch_tile_gemm(TileParams p, const void* operand, q8_dtype out_dtype,
                             cudaStream_t s);

// The forms for rows with a scale for each token (see TileForm): float outputs;
// the gated ones take N output channels and NB blocks of 128 packed rows, two
// rows a channel (see gated_rows); the last two f16 or bf16 alone.
enum Activation { kActNone, kActRelu, kActSilu, kActGelu };
cudaError_t launch_tile_token(TileParams p, const void* operand, q8_dtype out_dtype,
                              cudaStream_t s);
cudaError_t launch_tile_gated(TileParams p, const void* operand, q8_dtype out_dtype,
                              cudaStream_t s);
cudaError_t launch_tile_gated_grad(TileParams p, const void* operand, q8_dtype dtype,
                                   cudaStream_t s);
cudaError_t launch_tile_grad(TileParams p, const void* operand, q8_dtype dtype, cudaStream_t s);

// Rows of a packed gated weight: 16 of the gate, 16 of the up projection in
// turn, both padded with zeros to a multiple of 16 channels.
inline int64_t gated_rows(int64_t N) { return 2 * round_up(N, 16); }

// Weights [E][N][K] -> [E][NB][KB][4][128][16] bytes: for each block of 128
// output channels and 64 inputs, 16-input chunks of all 128 rows; top bits
// flipped, zeros beyond N and K.
cudaError_t launch_pack_tile_weight(const int8_t* w, int64_t E, int64_t N, int64_t K, uint8_t* dst,
                                    cudaStream_t s);
// *bound: the largest sum of |w| over 64 inputs (a k-block) in packed tiles.
cudaError_t launch_tile_weight_bound(const uint8_t* packed, int64_t tiles, int32_t* bound,
                                     cudaStream_t s);

// Token operand: dst[kb][s][64] = f16(x[row(s)][64 kb ..] - zp), zeros beyond
// K; row(s) = order[s] / k, or s when order is null; rows whose order is out
// of range are left alone.  Also zeroes `counts` (count_words of them).
struct OperandJob {
  const int8_t* x;
  int64_t x_rows, K;
  int R, k, KB, zp;
  const int32_t* order;
  uint4* dst;
  int32_t* counts;
  int count_words;
};
cudaError_t launch_tile_operand(const OperandJob& job, cudaStream_t s);

// Adapters A [L][r][K], B [L][N][r] (16-bit) and scaling [L] in the layouts
// the kernels read.
cudaError_t launch_pack_lora(const void* A, const void* B, const float* scaling, bool f16,
                             int64_t L, int64_t r, int64_t N, int64_t K, void* a_out, void* b_out,
                             float* s_out, cudaStream_t s);

// Everything the contraction with adapters needs before it, in one launch, two
// for sorted rows: the operand (op.k == 1; op.order null when the rows come as
// they are), each row's h, each row tile's adapters, and the rows' adapters in
// their order.
struct LoraJob {
  OperandJob op;
  const int32_t* adapter_ids;   // [R], in the order of x
  int L, r, rank16, tiles, list_stride;
  const uint16_t* a;            // packed A
  const float* scaling;
  float s_in;
  float* h;                     // [R][rank16 * 16], or blocks for MMAs (store_h)
  int TN;                       // rows of such a block, or 0
  int32_t* lists;
  int32_t* ids_out;             // [R] in sorted order, or null
  const int32_t* offsets;       // [L + 1] first sorted row of each adapter (with op.order)
  int shrink_ctas, list_ctas;   // set by the launcher
};
cudaError_t launch_lora_front(LoraJob job, bool f16, cudaStream_t s);

}  // namespace q8
