// api_tokens.cu -- the extern "C" entry points for rows with a scale for each
// token (declared at the end of include/q8ta.h): guards on the host, then the
// launches.
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "api_common.h"
#include "q8ta.h"
#include "tile_plan.h"
#include "token_internal.h"

namespace {

using namespace q8api;

bool float_type(q8_dtype dt) { return dt == Q8_F32 || dt == Q8_F16 || dt == Q8_BF16; }
bool half_type(q8_dtype dt) { return dt == Q8_F16 || dt == Q8_BF16; }
bool any_type(q8_dtype dt) { return float_type(dt) || dt == Q8_I8; }

// Rows and inputs of any call, and rows times outputs.
bool rows_ok(int64_t M, int64_t K) {
  return M >= 0 && M <= INT32_MAX && K >= 1 && K <= INT32_MAX / 2 && mul_ok(M, q8::round_up(K, 128) * 4);
}
bool outputs_ok(int64_t M, int64_t N) { return mul_ok(M, q8::round_up(N, 128) * 8); }

// act: "none", "relu" for the plain product; "silu", "gelu", "relu" for the gated.
int parse_gate(const char* a) {
  if (std::strcmp(a, "silu") == 0) return q8::kActSilu;
  if (std::strcmp(a, "gelu") == 0) return q8::kActGelu;
  if (std::strcmp(a, "relu") == 0) return q8::kActRelu;
  return -1;
}

constexpr int kMinRun = 4;   // k-blocks of a run at least

// The operand, parts and counts of a contraction, then the rows' scales.
struct TokenSpace {
  TilePlan plan;
  size_t scales, total;
};
TokenSpace token_space(const TilePlan& plan, int64_t M) {
  TokenSpace t{};
  t.plan = plan;
  t.scales = plan.total;
  t.total = t.scales + q8::align_ws(static_cast<size_t>(M) * 4);
  return t;
}
// (any height's plan has this size)
size_t token_space_bytes(int64_t M, int64_t K) { return token_space(plan_tiles(M, K, 1), M).total; }

// Inputs of the transposed gated weight: up to the end of the last block of 128
// packed rows, which is how far the gated gradient writes its operand.
int64_t gated_inputs(int64_t N) { return q8::round_up(q8::gated_rows(N), 128); }
bool gated_sizes_ok(int64_t N, int64_t K) {
  return N >= 1 && N <= (1 << 23) && tile_sizes_ok(1, q8::gated_rows(N), K) &&
         tile_sizes_ok(1, K, gated_inputs(N));
}

// Two contractions one after the other: the rows' operand and the gradients',
// one set of parts, both counts, each row's largest |dh| and power of two, and
// the largest scales and biases.
struct GradSpace {
  TilePlan rows, grads;
  size_t grad_operand, parts, counts, powers, total;
};
GradSpace gated_grad_space(const TilePlan& rows, const TilePlan& grads, int64_t M) {
  GradSpace t{};
  t.rows = rows;
  t.grads = grads;
  t.grad_operand = t.rows.operand;
  t.parts = t.grad_operand + t.grads.operand;
  t.counts = t.parts + t.grads.parts;
  t.powers = t.counts + 2 * t.grads.counts;
  t.total = t.powers + 2 * q8::align_ws(static_cast<size_t>(M) * 4) + q8::align_ws(16);
  return t;
}

q8::TileParams tile_params(int64_t M, int64_t N, int64_t rows, int64_t K, const TilePlan& plan,
                           const void* packed) {
  q8::TileParams p{};
  p.R = static_cast<int>(M);
  p.N = static_cast<int>(N);
  p.NB = static_cast<int>((rows + 127) / 128);
  p.KB = static_cast<int>((K + 63) / 64);
  p.E = 1;
  p.TN = plan.TN;
  p.max_tiles = static_cast<int>(max_tiles(M, 1, plan));
  p.grid = plan.grid;
  p.min_run = kMinRun;
  p.w = static_cast<const uint8_t*>(packed);
  p.w_bound = reinterpret_cast<const int32_t*>(p.w + tile_weight_bytes(1, rows, K));
  p.a_bound = a_bound_of(0);
  p.floor_f = -INFINITY;
  return p;
}

// Either form of rows: int8 ones with scales, or float ones to quantize.
q8_status check_rows(const void* x, q8_dtype x_dtype, const int8_t* x_q, const float* x_scales) {
  if (!x || (x_dtype == Q8_I8 && !x_scales)) return Q8_ERR_NULL;
  if (!aligned(x, q8::dtype_bytes(x_dtype)) || !aligned(x_scales, 4)) return Q8_ERR_ALIGN;
  return Q8_OK;
}

// The contraction's operand from either form.
cudaError_t make_operand(const void* x, q8_dtype x_dtype, int64_t M, int64_t K, int8_t* x_q,
                         float* scales, void* operand, int32_t* counts, int count_words,
                         cudaStream_t s) {
  const int KB = static_cast<int>((K + 63) / 64);
  if (x_dtype == Q8_I8) {
    q8::OperandJob job{};
    job.x = static_cast<const int8_t*>(x);
    job.x_rows = M;
    job.K = K;
    job.R = static_cast<int>(M);
    job.k = 1;
    job.KB = KB;
    job.dst = static_cast<uint4*>(operand);
    job.counts = counts;
    job.count_words = count_words;
    return q8::launch_tile_operand(job, s);
  }
  q8::QuantizeJob job{};
  job.x = x;
  job.M = M;
  job.K = K;
  job.q = x_q;
  job.scales = scales;
  job.operand = static_cast<uint16_t*>(operand);
  job.KB = KB;
  job.counts = counts;
  job.count_words = count_words;
  return q8::launch_quantize_token(job, x_dtype, s);
}

// linear_per_token and linear_gated once their own arguments are checked.
q8_status token_product(const void* x, q8_dtype x_dtype, int64_t M, int64_t K, int8_t* x_q,
                        float* x_scales, const void* packed, int64_t N, bool gated, int act,
                        const float* ws, const float* bias, q8_dtype out_dtype, void* out,
                        void* workspace, size_t workspace_bytes, cudaStream_t s) {
  q8_status st = check_rows(x, x_dtype, x_q, x_scales);
  if (st != Q8_OK) return st;
  if (!packed || !ws || !out) return Q8_ERR_NULL;
  if (!aligned(packed, q8::kWorkspaceAlign) || !aligned(ws, 4) || !aligned(bias, 4) ||
      !aligned(out, q8::dtype_bytes(out_dtype)))
    return Q8_ERR_ALIGN;
  const int64_t rows = gated ? q8::gated_rows(N) : N;
  if (q8::token_rows_fit(M, K, !gated && x_dtype == Q8_I8)) {
    q8::TokenRowsJob job{};
    job.x = x;
    job.x_dtype = x_dtype;
    job.M = M;
    job.K = K;
    job.q = x_q;
    job.scales = x_scales;
    job.w = static_cast<const uint8_t*>(packed);
    job.N = N;
    job.ws = ws;
    job.bias = bias;
    job.act = act;
    job.out_dtype = out_dtype;
    job.out = out;
    return cuda_status(q8::launch_token_rows(job, gated, s));
  }
  const TokenSpace sp = token_space(plan_group(M, rows, K, kMinRun), M);
  if (!units_ok(M, 1, rows, K, sp.plan)) return Q8_ERR_SHAPE;
  if (!workspace || workspace_bytes < sp.total) return Q8_ERR_WORKSPACE;
  if (!aligned(workspace, q8::kWorkspaceAlign)) return Q8_ERR_ALIGN;
  auto* space = static_cast<uint8_t*>(workspace);
  if (x_scales == nullptr) x_scales = reinterpret_cast<float*>(space + sp.scales);

  q8::TileParams p = tile_params(M, N, rows, K, sp.plan, packed);
  p.ws = ws;
  p.bias = bias;
  p.row_scale = x_scales;
  p.act = act;
  if (!gated && act == q8::kActRelu) p.floor_f = 0.0f;
  p.out = out;
  p.parts = reinterpret_cast<int32_t*>(space + sp.plan.operand);
  p.counts = reinterpret_cast<int32_t*>(space + sp.plan.operand + sp.plan.parts);
  cudaError_t e = make_operand(x, x_dtype, M, K, x_q, x_scales, space, p.counts,
                               p.grid * q8::kTileEpiWarps, s);
  if (e == cudaSuccess)
    e = gated ? q8::launch_tile_gated(p, space, out_dtype, s)
              : q8::launch_tile_token(p, space, out_dtype, s);
  return cuda_status(e);
}

}  // namespace

extern "C" {

q8_status q8_quantize_per_token(const void* x, q8_dtype dtype, int64_t M, int64_t K, int8_t* q,
                                float* scales, q8_stream_t stream) {
  if (!any_type(dtype)) return Q8_ERR_ARG;
  if (!float_type(dtype)) return Q8_ERR_UNSUPPORTED;
  if (!rows_ok(M, K)) return Q8_ERR_SHAPE;
  if (M == 0) return Q8_OK;
  if (!x || !q || !scales) return Q8_ERR_NULL;
  if (!aligned(x, q8::dtype_bytes(dtype)) || !aligned(scales, 4)) return Q8_ERR_ALIGN;
  q8::QuantizeJob job{};
  job.x = x;
  job.M = M;
  job.K = K;
  job.q = q;
  job.scales = scales;
  return cuda_status(q8::launch_quantize_token(job, dtype, cs(stream)));
}

q8_status q8_dequantize_per_token(const int8_t* q, const float* scales, int64_t M, int64_t K,
                                  q8_dtype dtype, void* out, q8_stream_t stream) {
  if (!any_type(dtype)) return Q8_ERR_ARG;
  if (!float_type(dtype)) return Q8_ERR_UNSUPPORTED;
  if (!rows_ok(M, K)) return Q8_ERR_SHAPE;
  if (M == 0) return Q8_OK;
  if (!q || !scales || !out) return Q8_ERR_NULL;
  if (!aligned(out, q8::dtype_bytes(dtype)) || !aligned(scales, 4)) return Q8_ERR_ALIGN;
  return cuda_status(q8::launch_dequantize_token(q, scales, M, K, dtype, out, cs(stream)));
}

// ---- products with scales for each token and channel ------------------------
size_t q8_linear_per_token_workspace_bytes(int64_t M, int64_t K, int64_t N) {
  // (for rows of any type)
  if (M < 1 || !rows_ok(M, K) || !tile_sizes_ok(1, N, K) || q8::token_rows_fit(M, K, false))
    return 0;
  return token_space_bytes(M, K);
}

q8_status q8_linear_per_token(const void* x, q8_dtype x_dtype, int64_t M, int64_t K, int8_t* x_q,
                              float* x_scales, const void* packed_weight, int64_t N,
                              const float* weight_scales, const float* bias,
                              const char* activation, q8_dtype out_dtype, void* out,
                              void* workspace, size_t workspace_bytes, q8_stream_t stream) {
  if (!activation) return Q8_ERR_NULL;
  if (!any_type(x_dtype) || !any_type(out_dtype)) return Q8_ERR_ARG;
  if (!float_type(out_dtype)) return Q8_ERR_UNSUPPORTED;
  if (!rows_ok(M, K) || !tile_sizes_ok(1, N, K) || !outputs_ok(M, N)) return Q8_ERR_SHAPE;
  const int relu = parse_activation(activation);
  if (relu < 0) return Q8_ERR_UNSUPPORTED;
  if (M == 0) return Q8_OK;
  return token_product(x, x_dtype, M, K, x_q, x_scales, packed_weight, N, false,
                       relu ? q8::kActRelu : q8::kActNone, weight_scales, bias, out_dtype, out,
                       workspace, workspace_bytes, cs(stream));
}

size_t q8_linear_per_token_backward_workspace_bytes(int64_t M, int64_t N, int64_t K) {
  if (M < 1 || !rows_ok(M, N) || !tile_sizes_ok(1, K, N)) return 0;
  return token_space_bytes(M, N);
}

q8_status q8_linear_per_token_backward(const void* dy, q8_dtype dtype, int64_t M, int64_t N,
                                       const void* y, const void* packed_transposed, int64_t K,
                                       const float* weight_scales, void* dx, void* workspace,
                                       size_t workspace_bytes, q8_stream_t stream) {
  if (!any_type(dtype)) return Q8_ERR_ARG;
  if (!half_type(dtype)) return Q8_ERR_UNSUPPORTED;
  if (!rows_ok(M, N) || !tile_sizes_ok(1, K, N) || !outputs_ok(M, K)) return Q8_ERR_SHAPE;
  if (M == 0) return Q8_OK;
  if (!dy || !packed_transposed || !weight_scales || !dx) return Q8_ERR_NULL;
  if (!aligned(dy, 2) || !aligned(y, 2) || !aligned(dx, 2) || !aligned(weight_scales, 4) ||
      !aligned(packed_transposed, q8::kWorkspaceAlign))
    return Q8_ERR_ALIGN;
  const TokenSpace sp = token_space(plan_group(M, K, N, kMinRun), M);
  if (!units_ok(M, 1, K, N, sp.plan)) return Q8_ERR_SHAPE;
  if (!workspace || workspace_bytes < sp.total) return Q8_ERR_WORKSPACE;
  if (!aligned(workspace, q8::kWorkspaceAlign)) return Q8_ERR_ALIGN;
  auto* space = static_cast<uint8_t*>(workspace);
  auto* unscale = reinterpret_cast<float*>(space + sp.scales);
  q8::TileParams p = tile_params(M, K, K, N, sp.plan, packed_transposed);
  p.out = dx;
  p.unscale = unscale;
  p.parts = reinterpret_cast<int32_t*>(space + sp.plan.operand);
  p.counts = reinterpret_cast<int32_t*>(space + sp.plan.operand + sp.plan.parts);
  q8::GradOperandJob job{};
  job.dy = dy;
  job.y = y;
  job.ws = weight_scales;
  job.M = M;
  job.N = N;
  job.dst = reinterpret_cast<uint16_t*>(space);
  job.unscale = unscale;
  job.KB = p.KB;
  job.counts = p.counts;
  job.count_words = p.grid * q8::kTileEpiWarps;
  cudaError_t e = q8::launch_grad_operand(job, dtype, cs(stream));
  if (e == cudaSuccess) e = q8::launch_tile_grad(p, space, dtype, cs(stream));
  return cuda_status(e);
}

// ---- the gated pair ---------------------------------------------------------
size_t q8_gated_packed_weight_bytes(int64_t N, int64_t K, int transposed) {
  if (!gated_sizes_ok(N, K)) return 0;
  return (transposed ? tile_weight_bytes(1, K, gated_inputs(N))
                     : tile_weight_bytes(1, q8::gated_rows(N), K)) +
         q8::kWorkspaceAlign;
}

q8_status q8_gated_pack_weight(const int8_t* gate, const int8_t* up, int64_t N, int64_t K,
                               int transposed, void* packed, size_t packed_bytes,
                               q8_stream_t stream) {
  if (!gate || !up || !packed) return Q8_ERR_NULL;
  if (!gated_sizes_ok(N, K)) return Q8_ERR_SHAPE;
  const size_t bytes = q8_gated_packed_weight_bytes(N, K, transposed);
  if (packed_bytes < bytes) return Q8_ERR_WORKSPACE;
  if (!aligned(packed, q8::kWorkspaceAlign)) return Q8_ERR_ALIGN;
  auto* dst = static_cast<uint8_t*>(packed);
  cudaError_t e = q8::launch_pack_gated(gate, up, N, K, transposed != 0, dst, cs(stream));
  // (the gradient's f32 sums need no bound)
  if (e == cudaSuccess && !transposed)
    e = q8::launch_tile_weight_bound(
        dst, static_cast<int64_t>((bytes - q8::kWorkspaceAlign) / 8192),
        reinterpret_cast<int32_t*>(dst + bytes - q8::kWorkspaceAlign), cs(stream));
  // finished before the call returns, as in q8_tile_pack_weight
  if (e == cudaSuccess) e = cudaStreamSynchronize(cs(stream));
  return cuda_status(e);
}

size_t q8_linear_gated_workspace_bytes(int64_t M, int64_t K, int64_t N) {
  if (M < 1 || !rows_ok(M, K) || !gated_sizes_ok(N, K) || q8::token_rows_fit(M, K, false))
    return 0;
  return token_space_bytes(M, K);
}

q8_status q8_linear_gated(const void* x, q8_dtype x_dtype, int64_t M, int64_t K, int8_t* x_q,
                          float* x_scales, const void* packed_weight, int64_t N,
                          const float* weight_scales, const float* bias, const char* activation,
                          q8_dtype out_dtype, void* out, void* workspace, size_t workspace_bytes,
                          q8_stream_t stream) {
  if (!activation) return Q8_ERR_NULL;
  if (!any_type(x_dtype) || !any_type(out_dtype)) return Q8_ERR_ARG;
  if (!float_type(out_dtype)) return Q8_ERR_UNSUPPORTED;
  if (!rows_ok(M, K) || !gated_sizes_ok(N, K) || !outputs_ok(M, 2 * N)) return Q8_ERR_SHAPE;
  const int act = parse_gate(activation);
  if (act < 0) return Q8_ERR_UNSUPPORTED;
  if (M == 0) return Q8_OK;
  return token_product(x, x_dtype, M, K, x_q, x_scales, packed_weight, N, true, act, weight_scales,
                       bias, out_dtype, out, workspace, workspace_bytes, cs(stream));
}

size_t q8_linear_gated_backward_workspace_bytes(int64_t M, int64_t K, int64_t N) {
  if (M < 1 || !rows_ok(M, K) || !gated_sizes_ok(N, K) || !rows_ok(M, gated_inputs(N))) return 0;
  return gated_grad_space(plan_tiles(M, K, 1), plan_tiles(M, gated_inputs(N), 1), M).total;
}

q8_status q8_linear_gated_backward(const void* dh, q8_dtype dtype, int64_t M, int64_t N,
                                   const int8_t* x_q, const float* x_scales, int64_t K,
                                   const void* packed_weight, const void* packed_transposed,
                                   const float* weight_scales, const float* bias,
                                   const char* activation, void* dx, void* workspace,
                                   size_t workspace_bytes, q8_stream_t stream) {
  if (!activation) return Q8_ERR_NULL;
  if (!any_type(dtype)) return Q8_ERR_ARG;
  if (!half_type(dtype)) return Q8_ERR_UNSUPPORTED;
  if (!rows_ok(M, K) || !gated_sizes_ok(N, K) || !rows_ok(M, gated_inputs(N)) ||
      !outputs_ok(M, 2 * N))
    return Q8_ERR_SHAPE;
  const int act = parse_gate(activation);
  if (act < 0) return Q8_ERR_UNSUPPORTED;
  if (M == 0) return Q8_OK;
  if (!dh || !x_q || !x_scales || !packed_weight || !packed_transposed || !weight_scales || !dx)
    return Q8_ERR_NULL;
  if (!aligned(dh, 2) || !aligned(dx, 2) || !aligned(x_scales, 4) || !aligned(weight_scales, 4) ||
      !aligned(bias, 4) || !aligned(packed_weight, q8::kWorkspaceAlign) ||
      !aligned(packed_transposed, q8::kWorkspaceAlign))
    return Q8_ERR_ALIGN;
  const int64_t rows = q8::gated_rows(N), inputs = gated_inputs(N);
  const GradSpace sp = gated_grad_space(plan_group(M, rows, K, kMinRun),
                                        plan_group(M, K, inputs, kMinRun), M);
  if (!units_ok(M, 1, rows, K, sp.rows) || !units_ok(M, 1, K, inputs, sp.grads)) return Q8_ERR_SHAPE;
  if (!workspace || workspace_bytes < sp.total) return Q8_ERR_WORKSPACE;
  if (!aligned(workspace, q8::kWorkspaceAlign)) return Q8_ERR_ALIGN;
  auto* space = static_cast<uint8_t*>(workspace);
  const size_t each = q8::align_ws(static_cast<size_t>(M) * 4);
  auto* most_dh = reinterpret_cast<float*>(space + sp.powers);
  auto* unscale = reinterpret_cast<float*>(space + sp.powers + each);
  auto* tops = reinterpret_cast<float*>(space + sp.powers + 2 * each);
  auto* counts = reinterpret_cast<int32_t*>(space + sp.counts);
  const int count_words = static_cast<int>(sp.grads.counts / 4);

  q8::TileParams p = tile_params(M, N, rows, K, sp.rows, packed_weight);
  p.ws = weight_scales;
  p.bias = bias;
  p.row_scale = x_scales;
  p.act = act;
  p.dh = dh;
  p.operand_out = reinterpret_cast<uint16_t*>(space + sp.grad_operand);
  p.K = K;
  p.most_dh = most_dh;
  p.tops = tops;
  p.unscale = unscale;
  p.parts = reinterpret_cast<int32_t*>(space + sp.parts);
  p.counts = counts;
  q8::TileParams g = tile_params(M, K, K, inputs, sp.grads, packed_transposed);
  g.out = dx;
  g.unscale = unscale;
  g.parts = p.parts;
  g.counts = counts + count_words;

  q8::GatedGradFrontJob job{};
  job.q = x_q;
  job.dh = dh;
  job.ws = weight_scales;
  job.bias = bias;
  job.M = M;
  job.N = N;
  job.K = K;
  job.operand = reinterpret_cast<uint16_t*>(space);
  job.KB = p.KB;
  job.most_dh = most_dh;
  job.tops = tops;
  job.counts = counts;
  job.count_words = 2 * count_words;
  cudaError_t e = q8::launch_gated_grad_front(job, dtype, cs(stream));
  if (e == cudaSuccess) e = q8::launch_tile_gated_grad(p, space, dtype, cs(stream));
  if (e == cudaSuccess) e = q8::launch_tile_grad(g, space + sp.grad_operand, dtype, cs(stream));
  return cuda_status(e);
}

}  // extern "C"
