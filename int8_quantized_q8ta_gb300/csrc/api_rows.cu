// api_rows.cu -- the extern "C" entry points for rows of one batch that go
// through different weights (declared at the end of include/q8ta.h): guards
// on the host, then the launches.
#include <cuda_runtime.h>

#include <cstdint>

#include "api_common.h"
#include "q8ta.h"
#include "rows_internal.h"

namespace {

using namespace q8api;

bool dtype_ok(q8_dtype dt) { return dt == Q8_F32 || dt == Q8_F16 || dt == Q8_BF16 || dt == Q8_I8; }

// Sizes of a routing problem and the alignment of its rows.
q8_status check_route(int64_t T, int64_t k, int64_t H, int64_t E) {
  if (T < 0 || k < 1 || H < 1 || E < 1 || E > q8::kMaxExperts) return Q8_ERR_SHAPE;
  if (!mul_ok(T, k) || T * k > INT32_MAX || !mul_ok(T * k, H) || !mul_ok(T * k * H, 4))
    return Q8_ERR_SHAPE;
  return Q8_OK;
}

bool aligned(const void* p, int64_t bytes) {
  return reinterpret_cast<uintptr_t>(p) % static_cast<uintptr_t>(bytes) == 0;
}

// ---- grouped int8 contraction ----------------------------------------------
size_t tile_weight_bytes(int64_t E, int64_t N, int64_t K) {
  return static_cast<size_t>(E) * ((N + 127) / 128) * ((K + 63) / 64) * 8192;
}

bool tile_sizes_ok(int64_t E, int64_t N, int64_t K) {
  return E >= 1 && E <= q8::kMaxExperts && N >= 1 && K >= 1 && N <= (1 << 24) &&
         K <= INT32_MAX / 2 && mul_ok(N, K) && mul_ok(E, N * K) && E * N * K <= INT64_MAX / 64;
}

// Tile height and grid of a problem of R rows in E groups.
struct TilePlan {
  int TN, grid;
  size_t operand, parts, counts, total;
};

// Adapters row by row in the epilogue, or by MMAs for each adapter and tile.
// Row by row costs a row's own dot products, a round of MMAs the same however
// few rows an adapter has.  Measured by row against by MMAs, ranks 16, 32
// adapters, K 4096: 64 rows x 11008 25.1 against 29.5 us, 192 rows x 4096 34.2
// against 42, x 11008 49.7 against 42.3; 4 adapters, 64 rows x 4096 17.3 both;
// 100 adapters, 512 rows x 11008 100 against 79, 300 rows x 8192 of K 2048 58
// against 44.  Over some sixty such sizes the best multiple is 7 (the chosen one
// 2.6% behind the faster on average); it sees neither N nor the row tiles, whose
// number is what makes row by row lose, and is up to 30% behind between 65 rows
// and 7 an adapter.
constexpr int kRowsPerAdapter = 7;
bool lora_by_row(int64_t M, int64_t L) { return M < kRowsPerAdapter * L; }

TilePlan plan_tiles(int64_t R, int64_t K, int64_t E, int64_t max_rows = q8::kMaxTileRows) {
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
int64_t max_tiles(int64_t R, int64_t E, const TilePlan& t) { return R / t.TN + std::min(E, R); }

// The k-blocks of all units are numbered in 32 bits.
bool units_ok(int64_t R, int64_t E, int64_t N, int64_t K, const TilePlan& t) {
  const int64_t tiles = max_tiles(R, E, t), blocks = (N + 127) / 128, kbs = (K + 63) / 64;
  return mul_ok(blocks, kbs) && mul_ok(tiles, blocks * kbs) && tiles * blocks * kbs <= INT32_MAX;
}

// ---- adapters --------------------------------------------------------------
bool lora_sizes_ok(int64_t L, int64_t N, int64_t K, int64_t r) {
  return L >= 1 && L <= q8::kMaxExperts && r >= 1 && r <= q8::kMaxRank && tile_sizes_ok(1, N, K);
}

// Packed adapters: B tiles, A rows, scaling (byte offsets).
struct LoraLayout {
  size_t a, scaling, total;
};
LoraLayout lora_layout(int64_t L, int64_t N, int64_t K, int64_t r) {
  const size_t rank16 = (r + 15) / 16;
  LoraLayout t{};
  t.a = static_cast<size_t>(L) * ((N + 127) / 128) * rank16 * 4096;
  t.scaling = t.a + static_cast<size_t>(L) * rank16 * 16 * q8::round_up(K, 64) * 2;
  t.total = q8::align_ws(t.scaling + static_cast<size_t>(L) * 4);
  return t;
}

// Workspace of the projection with adapters (byte offsets).
struct LoraSpace {
  TilePlan plan;
  size_t h, lists, sort, total;
};
LoraSpace lora_space(int64_t M, int64_t K, int64_t L, int64_t r) {
  LoraSpace t{};
  t.plan = plan_tiles(M, K, 1, lora_by_row(M, L) ? q8::kMaxByRow : q8::kMaxTileRows);
  const int64_t tiles = (M + t.plan.TN - 1) / t.plan.TN;
  t.h = t.plan.total;
  const size_t rank16 = (r + 15) / 16;
  t.lists = t.h + q8::align_ws(lora_by_row(M, L) ? static_cast<size_t>(M) * rank16 * 64
                                                 : static_cast<size_t>(tiles + L) * rank16 * t.plan.TN * 128);
  t.sort = t.lists + q8::align_ws(static_cast<size_t>(tiles) * (t.plan.TN + 1) * 4);
  t.total = t.sort + (tiles > 1 ? q8::align_ws((3 * static_cast<size_t>(M) + L + 1) * 4) : 0);
  return t;
}

// float rows (everything but the gather)
q8_status check_float(q8_dtype dt) {
  if (!dtype_ok(dt)) return Q8_ERR_ARG;
  return dt == Q8_I8 ? Q8_ERR_UNSUPPORTED : Q8_OK;
}

}  // namespace

extern "C" {

q8_status q8_expert_sort(const int32_t* expert_ids, int64_t T, int64_t k, int64_t E,
                         int32_t* order, int32_t* position, int32_t* offsets, q8_stream_t stream) {
  q8_status st = check_route(T, k, 1, E);
  if (st != Q8_OK) return st;
  if (!offsets || (T > 0 && (!expert_ids || !order || !position))) return Q8_ERR_NULL;
  if (!aligned(expert_ids, 4) || !aligned(order, 4) || !aligned(position, 4) ||
      !aligned(offsets, 4))
    return Q8_ERR_ALIGN;
  return cuda_status(q8::launch_expert_sort(expert_ids, T * k, static_cast<int>(E), order,
                                            position, offsets, cs(stream)));
}

q8_status q8_expert_gather(const void* x, q8_dtype dtype, int64_t T, int64_t k, int64_t H,
                           int64_t E, const int32_t* position, const int32_t* offsets, void* xs,
                           q8_stream_t stream) {
  if (!dtype_ok(dtype)) return Q8_ERR_ARG;
  q8_status st = check_route(T, k, H, E);
  if (st != Q8_OK) return st;
  if (T == 0) return Q8_OK;
  if (!x || !position || !offsets || !xs) return Q8_ERR_NULL;
  const int64_t b = q8::dtype_bytes(dtype);
  if (!aligned(x, b) || !aligned(xs, b) || !aligned(position, 4) || !aligned(offsets, 4))
    return Q8_ERR_ALIGN;
  return cuda_status(q8::launch_expert_gather(x, T, static_cast<int>(k), H * b, position, offsets,
                                              static_cast<int>(E), xs, cs(stream)));
}

q8_status q8_expert_dispatch(const void* x, q8_dtype dtype, int64_t T, int64_t H,
                             const int32_t* expert_ids, int64_t k, int64_t E, int32_t* order,
                             int32_t* position, int32_t* offsets, void* xs, q8_stream_t stream) {
  // every guard of both parts before anything is enqueued
  if (!dtype_ok(dtype)) return Q8_ERR_ARG;
  q8_status st = check_route(T, k, H, E);
  if (st != Q8_OK) return st;
  if (T > 0 && (!x || !xs)) return Q8_ERR_NULL;
  const int64_t b = q8::dtype_bytes(dtype);
  if (!aligned(x, b) || !aligned(xs, b)) return Q8_ERR_ALIGN;
  if (T == 0) return q8_expert_sort(expert_ids, T, k, E, order, position, offsets, stream);
  if (!expert_ids || !order || !position || !offsets) return Q8_ERR_NULL;
  if (!aligned(expert_ids, 4) || !aligned(order, 4) || !aligned(position, 4) ||
      !aligned(offsets, 4))
    return Q8_ERR_ALIGN;
  return cuda_status(q8::launch_expert_dispatch(x, T, static_cast<int>(k), H * b, expert_ids,
                                                static_cast<int>(E), order, position, offsets, xs,
                                                cs(stream)));
}

q8_status q8_expert_gather_backward(const void* dxs, q8_dtype dtype, int64_t T, int64_t k,
                                    int64_t H, const int32_t* position, void* dx,
                                    q8_stream_t stream) {
  q8_status st = check_float(dtype);
  if (st == Q8_OK) st = check_route(T, k, H, 1);
  if (st != Q8_OK) return st;
  if (T == 0) return Q8_OK;
  if (!dxs || !position || !dx) return Q8_ERR_NULL;
  const int64_t b = q8::dtype_bytes(dtype);
  if (!aligned(dxs, b) || !aligned(dx, b) || !aligned(position, 4)) return Q8_ERR_ALIGN;
  return cuda_status(q8::launch_expert_spread(dxs, dtype, nullptr, T, static_cast<int>(k), H,
                                              position, dx, cs(stream)));
}

q8_status q8_expert_combine(const void* z, q8_dtype dtype, const float* weights, int64_t T,
                            int64_t k, int64_t H, const int32_t* position, void* y,
                            q8_stream_t stream) {
  q8_status st = check_float(dtype);
  if (st == Q8_OK) st = check_route(T, k, H, 1);
  if (st != Q8_OK) return st;
  if (T == 0) return Q8_OK;
  if (!z || !weights || !position || !y) return Q8_ERR_NULL;
  const int64_t b = q8::dtype_bytes(dtype);
  if (!aligned(z, b) || !aligned(y, b) || !aligned(weights, 4) || !aligned(position, 4))
    return Q8_ERR_ALIGN;
  return cuda_status(q8::launch_expert_spread(z, dtype, weights, T, static_cast<int>(k), H,
                                              position, y, cs(stream)));
}

q8_status q8_expert_combine_backward(const void* dy, const void* z, q8_dtype dtype,
                                     const float* weights, int64_t T, int64_t k, int64_t H,
                                     int64_t E, const int32_t* position, const int32_t* offsets,
                                     void* dz, float* dweights, q8_stream_t stream) {
  q8_status st = check_float(dtype);
  if (st == Q8_OK) st = check_route(T, k, H, E);
  if (st != Q8_OK) return st;
  if (T == 0) return Q8_OK;
  if (!dy || !z || !weights || !position || !offsets || !dz || !dweights) return Q8_ERR_NULL;
  const int64_t b = q8::dtype_bytes(dtype);
  if (!aligned(dy, b) || !aligned(z, b) || !aligned(dz, b) || !aligned(weights, 4) ||
      !aligned(dweights, 4) || !aligned(position, 4) || !aligned(offsets, 4))
    return Q8_ERR_ALIGN;
  return cuda_status(q8::launch_expert_combine_bwd(dy, z, dtype, weights, T, static_cast<int>(k),
                                                   H, position, offsets, static_cast<int>(E), dz,
                                                   dweights, cs(stream)));
}

size_t q8_tile_packed_weight_bytes(int64_t E, int64_t N, int64_t K) {
  return tile_sizes_ok(E, N, K) ? tile_weight_bytes(E, N, K) + q8::kWorkspaceAlign : 0;
}

q8_status q8_tile_pack_weight(const int8_t* weight, int64_t E, int64_t N, int64_t K, void* packed,
                              size_t packed_bytes, q8_stream_t stream) {
  if (!weight || !packed) return Q8_ERR_NULL;
  if (!tile_sizes_ok(E, N, K)) return Q8_ERR_SHAPE;
  if (packed_bytes < q8_tile_packed_weight_bytes(E, N, K)) return Q8_ERR_WORKSPACE;
  if (!aligned(packed, q8::kWorkspaceAlign)) return Q8_ERR_ALIGN;
  auto* dst = static_cast<uint8_t*>(packed);
  cudaError_t e = q8::launch_pack_tile_weight(weight, E, N, K, dst, cs(stream));
  if (e == cudaSuccess)
    e = q8::launch_weight_block_bound(weight, E * N, K, 1, K,
                                      reinterpret_cast<int32_t*>(dst + tile_weight_bytes(E, N, K)),
                                      cs(stream));
  // finished before the call returns: later kernels read a packed weight
  // without waiting for the kernel before them
  if (e == cudaSuccess) e = cudaStreamSynchronize(cs(stream));
  return cuda_status(e);
}

size_t q8_linear_experts_workspace_bytes(int64_t R, int64_t K, int64_t E) {
  if (R < 1 || R > INT32_MAX || K < 1 || K > INT32_MAX / 2 || E < 1 || E > q8::kMaxExperts)
    return 0;
  return plan_tiles(R, K, E).total;
}

q8_status q8_linear_experts(const int8_t* x, int x_sorted, int64_t T, int64_t k, int64_t K,
                            double input_scale, int32_t input_zero_point,
                            const void* packed_weight, int64_t E, int64_t N,
                            const float* weight_scales, const float* bias, const int32_t* order,
                            const int32_t* offsets, double output_scale,
                            int32_t output_zero_point, const char* activation, q8_dtype out_dtype,
                            void* out, void* workspace, size_t workspace_bytes,
                            q8_stream_t stream) {
  if (!activation) return Q8_ERR_NULL;
  if (!dtype_ok(out_dtype)) return Q8_ERR_ARG;
  q8_status st = check_route(T, k, 1, E);
  if (st != Q8_OK) return st;
  if (!tile_sizes_ok(E, N, K)) return Q8_ERR_SHAPE;
  const int64_t R = T * k;
  if (!mul_ok(R, q8::round_up(K, 64) * 2) || !mul_ok(R, N * 4)) return Q8_ERR_SHAPE;
  const int relu = parse_activation(activation);
  if (relu < 0) return Q8_ERR_UNSUPPORTED;
  if (!scale_ok(input_scale) || !scale_ok(output_scale) || !zp_ok(input_zero_point) ||
      !zp_ok(output_zero_point))
    return Q8_ERR_ARG;
  if (R == 0) return Q8_OK;
  if (!x || !packed_weight || !weight_scales || !order || !offsets || !out) return Q8_ERR_NULL;
  if (!aligned(packed_weight, q8::kWorkspaceAlign) || !aligned(weight_scales, 4) ||
      !aligned(bias, 4) || !aligned(order, 4) || !aligned(offsets, 4) ||
      !aligned(out, q8::dtype_bytes(out_dtype)))
    return Q8_ERR_ALIGN;
  const TilePlan plan = plan_tiles(R, K, E);
  if (!units_ok(R, E, N, K, plan)) return Q8_ERR_SHAPE;
  if (!workspace || workspace_bytes < plan.total) return Q8_ERR_WORKSPACE;
  if (!aligned(workspace, q8::kWorkspaceAlign)) return Q8_ERR_ALIGN;
  auto* ws = static_cast<uint8_t*>(workspace);

  q8::TileParams p{};
  p.R = static_cast<int>(R);
  p.N = static_cast<int>(N);
  p.NB = static_cast<int>((N + 127) / 128);
  p.KB = static_cast<int>((K + 63) / 64);
  p.E = static_cast<int>(E);
  p.offsets = offsets;
  p.TN = plan.TN;
  p.max_tiles = static_cast<int>(max_tiles(R, E, plan));
  p.grid = plan.grid;
  p.min_run = 4;
  p.w = static_cast<const uint8_t*>(packed_weight);
  p.w_bound = reinterpret_cast<const int32_t*>(p.w + tile_weight_bytes(E, N, K));
  p.a_bound = a_bound_of(input_zero_point);
  p.ws = weight_scales;
  p.bias = bias;
  p.rq = make_rq(input_scale, output_scale, output_zero_point, relu);
  p.floor_f = relu ? 0.0f : -INFINITY;
  p.out = out;
  p.parts = reinterpret_cast<int32_t*>(ws + plan.operand);
  p.counts = reinterpret_cast<int32_t*>(ws + plan.operand + plan.parts);

  q8::OperandJob job{};
  job.x = x;
  job.x_rows = x_sorted ? R : T;
  job.K = K;
  job.R = p.R;
  job.k = static_cast<int>(k);
  job.KB = p.KB;
  job.zp = input_zero_point;
  job.order = x_sorted ? nullptr : order;
  job.dst = reinterpret_cast<uint4*>(ws);
  job.counts = p.counts;
  job.count_words = plan.grid * q8::kTileEpiWarps;
  cudaError_t e = q8::launch_tile_operand(job, cs(stream));
  if (e == cudaSuccess) e = q8::launch_tile_gemm(p, ws, out_dtype, cs(stream));
  return cuda_status(e);
}

// ---- low-rank adapters beside a shared projection ---------------------------
size_t q8_lora_packed_bytes(int64_t L, int64_t N, int64_t K, int64_t r) {
  return lora_sizes_ok(L, N, K, r) ? lora_layout(L, N, K, r).total : 0;
}

q8_status q8_lora_pack(const void* A, const void* B, const float* scaling, q8_dtype dtype,
                       int64_t L, int64_t r, int64_t N, int64_t K, void* packed,
                       size_t packed_bytes, q8_stream_t stream) {
  if (!A || !B || !scaling || !packed) return Q8_ERR_NULL;
  if (!dtype_ok(dtype)) return Q8_ERR_ARG;
  if (dtype != Q8_F16 && dtype != Q8_BF16) return Q8_ERR_UNSUPPORTED;
  if (!lora_sizes_ok(L, N, K, r)) return Q8_ERR_SHAPE;
  const LoraLayout lay = lora_layout(L, N, K, r);
  if (packed_bytes < lay.total) return Q8_ERR_WORKSPACE;
  if (!aligned(packed, q8::kWorkspaceAlign) || !aligned(A, 2) || !aligned(B, 2) ||
      !aligned(scaling, 4))
    return Q8_ERR_ALIGN;
  auto* dst = static_cast<uint8_t*>(packed);
  cudaError_t e = q8::launch_pack_lora(A, B, scaling, dtype == Q8_F16, L, r, N, K, dst + lay.a, dst,
                                       reinterpret_cast<float*>(dst + lay.scaling), cs(stream));
  if (e == cudaSuccess) e = cudaStreamSynchronize(cs(stream));   // load time, as for weights
  return cuda_status(e);
}

size_t q8_linear_lora_workspace_bytes(int64_t M, int64_t K, int64_t L, int64_t r) {
  if (M < 1 || M > INT32_MAX || K < 1 || K > INT32_MAX / 2 || L < 1 || L > q8::kMaxExperts ||
      r < 1 || r > q8::kMaxRank)
    return 0;
  return lora_space(M, K, L, r).total;
}

q8_status q8_linear_lora(const int8_t* x, int64_t M, int64_t K, double input_scale,
                         int32_t input_zero_point, const void* packed_weight, int64_t N,
                         const float* weight_scales, const float* bias, const void* packed_lora,
                         q8_dtype lora_dtype, int64_t L, int64_t r, const int32_t* adapter_ids,
                         double output_scale, int32_t output_zero_point, const char* activation,
                         q8_dtype out_dtype, void* out, void* workspace, size_t workspace_bytes,
                         q8_stream_t stream) {
  if (!activation) return Q8_ERR_NULL;
  if (!dtype_ok(out_dtype) || !dtype_ok(lora_dtype)) return Q8_ERR_ARG;
  if (lora_dtype != Q8_F16 && lora_dtype != Q8_BF16) return Q8_ERR_UNSUPPORTED;
  if (M < 0 || M > INT32_MAX || !lora_sizes_ok(L, N, K, r)) return Q8_ERR_SHAPE;
  if (!mul_ok(M, q8::round_up(K, 64) * 2) || !mul_ok(M, N * 4)) return Q8_ERR_SHAPE;
  const int relu = parse_activation(activation);
  if (relu < 0) return Q8_ERR_UNSUPPORTED;
  if (!scale_ok(input_scale) || !scale_ok(output_scale) || !zp_ok(input_zero_point) ||
      !zp_ok(output_zero_point))
    return Q8_ERR_ARG;
  if (M == 0) return Q8_OK;
  if (!x || !packed_weight || !weight_scales || !packed_lora || !adapter_ids || !out)
    return Q8_ERR_NULL;
  if (!aligned(packed_weight, q8::kWorkspaceAlign) || !aligned(packed_lora, q8::kWorkspaceAlign) ||
      !aligned(weight_scales, 4) || !aligned(bias, 4) || !aligned(adapter_ids, 4) ||
      !aligned(out, q8::dtype_bytes(out_dtype)))
    return Q8_ERR_ALIGN;
  const LoraSpace sp = lora_space(M, K, L, r);
  if (!units_ok(M, 1, N, K, sp.plan)) return Q8_ERR_SHAPE;
  if ((M / 32 + q8::kMaxTileRows) * ((r + 15) / 16) > INT32_MAX / 16) return Q8_ERR_SHAPE;
  if (!workspace || workspace_bytes < sp.total) return Q8_ERR_WORKSPACE;
  if (!aligned(workspace, q8::kWorkspaceAlign)) return Q8_ERR_ALIGN;
  auto* ws = static_cast<uint8_t*>(workspace);
  const LoraLayout lay = lora_layout(L, N, K, r);
  const auto* lora = static_cast<const uint8_t*>(packed_lora);

  q8::TileParams p{};
  p.R = static_cast<int>(M);
  p.N = static_cast<int>(N);
  p.NB = static_cast<int>((N + 127) / 128);
  p.KB = static_cast<int>((K + 63) / 64);
  p.E = 1;
  p.TN = sp.plan.TN;
  p.max_tiles = static_cast<int>(max_tiles(M, 1, sp.plan));
  p.grid = sp.plan.grid;
  p.min_run = 4;
  p.w = static_cast<const uint8_t*>(packed_weight);
  p.w_bound = reinterpret_cast<const int32_t*>(p.w + tile_weight_bytes(1, N, K));
  p.a_bound = a_bound_of(input_zero_point);
  p.ws = weight_scales;
  p.bias = bias;
  p.rq = make_rq(input_scale, output_scale, output_zero_point, relu);
  p.floor_f = relu ? 0.0f : -INFINITY;
  p.out = out;
  p.parts = reinterpret_cast<int32_t*>(ws + sp.plan.operand);
  p.counts = reinterpret_cast<int32_t*>(ws + sp.plan.operand + sp.plan.parts);
  p.L = static_cast<int>(L);
  p.rank16 = static_cast<int>((r + 15) / 16);
  p.lora_f16 = lora_dtype == Q8_F16;
  p.by_row = lora_by_row(M, L);
  p.lora_b = lora;
  p.h = reinterpret_cast<const float*>(ws + sp.h);
  p.lists = reinterpret_cast<const int32_t*>(ws + sp.lists);
  p.list_stride = p.TN + 1;

  q8::LoraJob job{};
  job.op.x = x;
  job.op.x_rows = M;
  job.op.K = K;
  job.op.R = p.R;
  job.op.k = 1;
  job.op.KB = p.KB;
  job.op.zp = input_zero_point;
  job.op.dst = reinterpret_cast<uint4*>(ws);
  job.op.counts = p.counts;
  job.op.count_words = p.grid * q8::kTileEpiWarps;
  job.adapter_ids = adapter_ids;
  job.L = p.L;
  job.r = static_cast<int>(r);
  job.rank16 = p.rank16;
  job.tiles = (p.R + p.TN - 1) / p.TN;
  job.list_stride = p.list_stride;
  job.a = reinterpret_cast<const uint16_t*>(lora + lay.a);
  job.scaling = reinterpret_cast<const float*>(lora + lay.scaling);
  job.s_in = static_cast<float>(input_scale);
  job.h = reinterpret_cast<float*>(ws + sp.h);
  job.TN = p.by_row ? 0 : p.TN;
  job.lists = reinterpret_cast<int32_t*>(ws + sp.lists);
  cudaError_t e = cudaSuccess;
  if (job.tiles == 1) {
    p.ids = adapter_ids;
  } else {
    // several row tiles: rows sorted by adapter, so that a tile meets few
    auto* sorted = reinterpret_cast<int32_t*>(ws + sp.sort);
    int32_t *order = sorted, *position = sorted + M, *ids = sorted + 2 * M,
            *offsets = sorted + 3 * M;
    e = q8::launch_expert_sort(adapter_ids, M, p.L, order, position, offsets, cs(stream), true);
    job.op.order = order;
    job.offsets = offsets;
    job.ids_out = ids;
    p.ids = ids;
    p.out_rows = order;
  }
  if (e == cudaSuccess) e = q8::launch_lora_front(job, lora_dtype == Q8_F16, cs(stream));
  if (e == cudaSuccess) e = q8::launch_tile_gemm(p, ws, out_dtype, cs(stream));
  return cuda_status(e);
}

}  // extern "C"
