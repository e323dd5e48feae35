// token_device.cuh -- device helpers of the operators for rows with a scale for
// each token: loads and stores by float type, a row's scale, its integers.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cfloat>
#include <cstdint>

#include "q8ta.h"
#include "rows_internal.h"
#include "tile_device.cuh"

namespace q8 {

// 16-bit floats by their type (Q8_F16 or Q8_BF16).
template <int DT>
__device__ __forceinline__ float half_bits_to_float(uint32_t v) {
  if constexpr (DT == Q8_F16) return __half2float(__ushort_as_half(static_cast<uint16_t>(v)));
  else return __uint_as_float(v << 16);
}
template <int DT>
__device__ __forceinline__ uint32_t float_to_half_bits(float v) {
  if constexpr (DT == Q8_F16) return __half_as_ushort(__float2half_rn(v));
  else return __bfloat16_as_ushort(__float2bfloat16_rn(v));
}

// All ones in each half of a word where its 16-bit float is above 0.  (Positive
// numbers and infinity have encodings from 1 to infinity's; NaN's are above.)
template <int DT>
__device__ __forceinline__ uint32_t above_zero(uint32_t v) {
  constexpr uint32_t kInf = DT == Q8_F16 ? 0x7c007c00u : 0x7f807f80u;
  return __vcmpgts2(v, 0u) & __vcmpleu2(v, kInf);
}

template <int DT>
__device__ __forceinline__ void store_one(void* out, int64_t i, float v) {
  if constexpr (DT == Q8_F32) static_cast<float*>(out)[i] = v;
  else static_cast<uint16_t*>(out)[i] = static_cast<uint16_t>(float_to_half_bits<DT>(v));
}
// Eight values at element i (a multiple of 8 on a 16-byte aligned base).
template <int DT>
__device__ __forceinline__ void store_x8(void* out, int64_t i, const float (&v)[8]) {
  if constexpr (DT == Q8_F32) {
    auto* to = reinterpret_cast<float4*>(static_cast<float*>(out) + i);
    to[0] = make_float4(v[0], v[1], v[2], v[3]);
    to[1] = make_float4(v[4], v[5], v[6], v[7]);
  } else {
    uint32_t r[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
      r[j] = float_to_half_bits<DT>(v[2 * j]) | (float_to_half_bits<DT>(v[2 * j + 1]) << 16);
    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(out) + i) = make_uint4(r[0], r[1], r[2], r[3]);
  }
}
// (Rows that an earlier kernel may have written are read with ordinary loads.)
// Eight 16-bit values of a row from column n0 on, zeros from column n on.
template <bool VEC>
__device__ __forceinline__ uint4 load_halves(const uint16_t* p, int64_t row, int64_t n0, int64_t n) {
  if constexpr (VEC)
    return n0 < n ? *reinterpret_cast<const uint4*>(p + row + n0) : make_uint4(0, 0, 0, 0);
  uint32_t v[4] = {0, 0, 0, 0};
#pragma unroll
  for (int j = 0; j < 8; ++j)
    if (n0 + j < n) v[j / 2] |= static_cast<uint32_t>(p[row + n0 + j]) << (16 * (j & 1));
  return make_uint4(v[0], v[1], v[2], v[3]);
}

// A row's scale from the encoding of its largest magnitude (of NaN where the
// row holds one: their encodings are above infinity's), and the scale's
// reciprocal.  Both are the correctly rounded f32 quotients that
// q8_quantize_per_tensor would be given and form ((float)(1.0 / (double)s)
// rounds 1 / s twice, but never to another float: s times a number of 25 bits
// has 49 at most, so 1 / s is no nearer than 2^-49 to a midpoint).  Scales
// below f32's normal numbers have no finite reciprocal: such rows count as
// zeros.
struct TokenScale {
  float scale, inv;
};
__device__ __forceinline__ TokenScale token_scale(uint32_t top) {
  TokenScale t;
  t.scale = __fdiv_rn(__uint_as_float(top), 127.0f);
  t.inv = __frcp_rn(t.scale);
  if (t.scale < FLT_MIN) t.scale = t.inv = 0.0f;
  return t;
}
// The byte of rint(x * inv), |x * inv| < 128 (the low byte of the sum's
// encoding; see round_add_clamp_i).  Infinities and NaN give some byte: their
// row's scale is not finite.
__device__ __forceinline__ uint32_t token_byte(float x, float inv) {
  return __float_as_uint(__fadd_rn(__fmul_rn(x, inv), kRoundMagic));
}
__device__ __forceinline__ uint32_t four_bytes(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  return __byte_perm(__byte_perm(a, b, 0x0040), __byte_perm(c, d, 0x0040), 0x5410);
}
// Eight int8 values in f16 (exact).
__device__ __forceinline__ uint4 token_f16x8(uint2 w) {
  const __half2 minus = __halves2half2(__ushort_as_half(0x6480), __ushort_as_half(0x6480));
  w.x ^= 0x80808080u;
  w.y ^= 0x80808080u;
  return make_uint4(biased_to_f16x2(w.x, 0x4140, minus), biased_to_f16x2(w.x, 0x4342, minus),
                    biased_to_f16x2(w.y, 0x4140, minus), biased_to_f16x2(w.y, 0x4342, minus));
}

// v of one exact sum: the row's scale, the channel's, the bias, one rounding a
// step.
__device__ __forceinline__ float token_value(int32_t acc, float s, float ws, float b) {
  return __fadd_rn(__fmul_rn(__fmul_rn(__int2float_rn(acc), s), ws), b);
}

// act(g), and with GRAD act'(g) too.  exp and the division are the fast ones (a
// few units in the last place of f32); both run into 0 or infinity where the
// sigmoid does.
template <bool GRAD>
__device__ __forceinline__ float activate(float g, int act, float& slope) {
  if (act == kActSilu) {
    const float sigma = __fdividef(1.0f, 1.0f + __expf(-g));
    const float a = g * sigma;
    if constexpr (GRAD) slope = fmaf(a, 1.0f - sigma, sigma);
    return a;
  }
  if (act == kActGelu) {
    const float phi = fmaf(0.5f, erff(g * 0.70710678f), 0.5f);
    if constexpr (GRAD) slope = fmaf(g * 0.39894228f, __expf(-0.5f * g * g), phi);
    return g * phi;
  }
  if constexpr (GRAD) slope = g > 0.0f ? 1.0f : 0.0f;
  return max_nan(g, 0.0f);
}
// No |act'| is above this (silu's reaches 1.10, gelu's 1.13).
constexpr float kSteepest = 1.25f;

// Gradients go into their product as f16 numbers, whatever their type: 11 bits,
// where bf16 has 8.  Each row is multiplied by a power of two that puts a bound
// on its values between 2^14 and 2^15, so that f16's few exponents reach 29
// powers of two below that bound, and the row's sums are divided by it again,
// exactly.  (Beyond 2^126 either way the row keeps what f32 can do.)
struct RowPower {
  float rescale, unscale;
};
__device__ __forceinline__ RowPower row_power(float bound) {
  const int exponent = static_cast<int>(__float_as_uint(bound) >> 23) & 255;
  // (zeros, infinities and NaN: as they are)
  const int e = exponent == 0 || exponent == 255 ? 0 : min(126, max(-126, 127 + 14 - exponent));
  return {__uint_as_float(static_cast<uint32_t>(127 + e) << 23),
          __uint_as_float(static_cast<uint32_t>(127 - e) << 23)};
}
__device__ __forceinline__ uint16_t grad_bits(float v) {
  return __half_as_ushort(__float2half_rn(v));
}

// What a thread loads of a row at once: 8 values on 16-byte boundaries, or one.
template <int DT, bool VEC>
struct TokenItem;

template <int DT>
struct TokenItem<DT, true> {
  static constexpr int kWidth = 8;
  static constexpr int kWords = DT == Q8_F32 ? 8 : 4;
  uint32_t w[kWords];
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int j = 0; j < kWords; ++j) w[j] = 0;
  }
  __device__ __forceinline__ void load(const void* x, int64_t i) {
    const auto* p = reinterpret_cast<const uint4*>(
        static_cast<const uint8_t*>(x) + i * (DT == Q8_F32 ? 4 : 2));
#pragma unroll
    for (int j = 0; j < kWords / 4; ++j) {
      const uint4 v = p[j];
      w[j * 4] = v.x;
      w[j * 4 + 1] = v.y;
      w[j * 4 + 2] = v.z;
      w[j * 4 + 3] = v.w;
    }
  }
  __device__ __forceinline__ float value(int j) const {
    if constexpr (DT == Q8_F32) return __uint_as_float(w[j]);
    else return half_bits_to_float<DT>((j & 1) ? w[j / 2] >> 16 : w[j / 2] & 0xffffu);
  }
  // The encoding of the largest magnitude, in f32 (magnitudes order like their
  // encodings).
  __device__ __forceinline__ uint32_t top() const {
    if constexpr (DT == Q8_F32) {
      uint32_t t = 0;
#pragma unroll
      for (int j = 0; j < 8; ++j) t = max(t, w[j] & 0x7fffffffu);
      return t;
    } else {
      uint32_t t = 0;
#pragma unroll
      for (int j = 0; j < 4; ++j) t = __vmaxu2(t, w[j] & 0x7fff7fffu);
      return __float_as_uint(half_bits_to_float<DT>(max(t & 0xffffu, t >> 16)));
    }
  }
  __device__ __forceinline__ uint2 quantize(float inv) const {
    uint32_t b[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) b[j] = token_byte(value(j), inv);
    return make_uint2(four_bytes(b[0], b[1], b[2], b[3]), four_bytes(b[4], b[5], b[6], b[7]));
  }
};

template <int DT>
struct TokenItem<DT, false> {
  static constexpr int kWidth = 1;
  float v;
  __device__ __forceinline__ void zero() { v = 0.0f; }
  __device__ __forceinline__ void load(const void* x, int64_t i) {
    if constexpr (DT == Q8_F32) v = static_cast<const float*>(x)[i];
    else v = half_bits_to_float<DT>(static_cast<const uint16_t*>(x)[i]);
  }
  __device__ __forceinline__ uint32_t top() const { return __float_as_uint(v) & 0x7fffffffu; }
  __device__ __forceinline__ int8_t quantize(float inv) const {
    return static_cast<int8_t>(token_byte(v, inv));
  }
};

}  // namespace q8
