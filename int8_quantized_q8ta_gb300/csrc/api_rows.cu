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
  st = q8_expert_sort(expert_ids, T, k, E, order, position, offsets, stream);
  if (st != Q8_OK) return st;
  return q8_expert_gather(x, dtype, T, k, H, E, position, offsets, xs, stream);
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

}  // extern "C"
