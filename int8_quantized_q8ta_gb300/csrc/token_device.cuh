// token_device.cuh -- device helpers of the operators for rows with a scale for
// each token: loads and stores by float type, a row's scale, its integers.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cfloat>
#include <cstdint>
#include <type_traits>

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
// ---------------------------------------------------------------------------
// Rows of any length, so that begin anywhere: what a thread wants of one, 8
// values, comes as the aligned 16 bytes that hold it and is shifted into place
// once it has arrived.  (Rows that an earlier kernel may have written are read
// with ordinary loads.)
// ---------------------------------------------------------------------------

// The bytes of a matrix, and where one of its rows begins.
struct RowBytes {
  const uint8_t *lo, *hi, *at;
};
template <typename T>
__device__ __forceinline__ RowBytes row_bytes(const void* x, int64_t M, int64_t K, int64_t m) {
  const auto* lo = static_cast<const uint8_t*>(x);
  return {lo, lo + M * K * static_cast<int64_t>(sizeof(T)), lo + m * K * static_cast<int64_t>(sizeof(T))};
}

// The 16 bytes at a 16-byte boundary, zeros outside [lo, hi).  All loads are in
// flight together: a matrix's last item comes here, and the kernel waits for it.
__device__ __forceinline__ uint4 load_within(const uint8_t* p, const uint8_t* lo, const uint8_t* hi) {
  uint32_t v[4] = {0, 0, 0, 0};
  const auto* p2 = reinterpret_cast<const uint16_t*>(p);   // (elements are two bytes or four)
#pragma unroll
  for (int j = 0; j < 8; ++j)
    if (p + 2 * j >= lo && p + 2 * j < hi)
      v[j >> 1] |= static_cast<uint32_t>(p2[j]) << (16 * (j & 1));
  return make_uint4(v[0], v[1], v[2], v[3]);
}

// W words from byte s < 16 of W + 4.
template <int W>
__device__ __forceinline__ void shift_words(uint32_t (&w)[W + 4], uint32_t s) {
  if (s & 8) {
#pragma unroll
    for (int j = 0; j < W + 2; ++j) w[j] = w[j + 2];
  }
  if (s & 4) {
#pragma unroll
    for (int j = 0; j < W + 1; ++j) w[j] = w[j + 1];
  }
  if (s & 3) {
#pragma unroll
    for (int j = 0; j < W; ++j) w[j] = __funnelshift_r(w[j], w[j + 1], (s & 3) * 8);
  }
}

// 32 W bits of a row: `load` asks for them, `settle` puts them in w[0 .. W - 1],
// zeros from `bytes` on.  VEC: the row begins on 16 bytes and is a multiple of
// them.
template <int W, bool VEC>
struct RowItem {
  uint32_t w[W + (VEC ? 0 : 4)];
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int j = 0; j < W + (VEC ? 0 : 4); ++j) w[j] = 0;
  }
  // item c of the row, of `bytes` in all
  __device__ __forceinline__ void load(const RowBytes& row, int64_t c, int64_t bytes) {
    const uint8_t* p = row.at + c * (W * 4);
    zero();
    if constexpr (VEC) {
      if (c * (W * 4) < bytes)
#pragma unroll
        for (int j = 0; j < W; j += 4) put(j, *reinterpret_cast<const uint4*>(p + j * 4));
    } else if (c * (W * 4) < bytes) {
      const uint32_t s = reinterpret_cast<uintptr_t>(p) & 15;
      p -= s;
      if (p >= row.lo && p + (W * 4 + 16) <= row.hi) {
#pragma unroll
        for (int j = 0; j <= W; j += 4) put(j, *reinterpret_cast<const uint4*>(p + j * 4));
      } else {   // the ends of the matrix
#pragma unroll
        for (int j = 0; j <= W; j += 4) put(j, load_within(p + j * 4, row.lo, row.hi));
      }
    }
  }
  __device__ __forceinline__ void settle(const RowBytes& row, int64_t c, int64_t bytes) {
    if constexpr (!VEC) {
      const int64_t left = bytes - c * (W * 4);
      if (left <= 0) return;   // zeros
      shift_words<W>(w, static_cast<uint32_t>(reinterpret_cast<uintptr_t>(row.at) + c * (W * 4)) & 15);
      if (left < W * 4) {
#pragma unroll
        for (int j = 0; j < W; ++j) {
          const int n = static_cast<int>(left) - j * 4;   // bytes of this word
          if (n < 4) w[j] &= n <= 0 ? 0u : (1u << (8 * n)) - 1;
        }
      }
    }
  }

 private:
  __device__ __forceinline__ void put(int j, const uint4& v) {
    w[j] = v.x;
    w[j + 1] = v.y;
    w[j + 2] = v.z;
    w[j + 3] = v.w;
  }
};

// Eight int8 values from any byte on: two aligned words of 8 bytes.
template <bool VEC>
__device__ __forceinline__ uint2 load_int8x8(const int8_t* q, int64_t row, int64_t k0, int64_t K,
                                             const int8_t* end) {
  if (k0 >= K) return make_uint2(0, 0);
  const int8_t* p = q + row + k0;
  if constexpr (VEC) return *reinterpret_cast<const uint2*>(p);
  const uint32_t s = reinterpret_cast<uintptr_t>(p) & 7;
  const int8_t* p0 = p - s;
  const auto part = [&](const int8_t* a) {
    if (a >= q && a + 8 <= end) return *reinterpret_cast<const uint64_t*>(a);
    uint64_t v = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (a + j >= q && a + j < end) v |= static_cast<uint64_t>(static_cast<uint8_t>(a[j])) << (8 * j);
    return v;
  };
  uint64_t v = part(p0) >> (8 * s);
  if (s != 0) v |= part(p0 + 8) << (64 - 8 * s);
  if (K - k0 < 8) v &= (uint64_t{1} << (8 * (K - k0))) - 1;
  return make_uint2(static_cast<uint32_t>(v), static_cast<uint32_t>(v >> 32));
}

// The first n bytes of each lane's 8 go to p, where lane l's p is lane 0's + 8 l
// (p of any alignment; lanes without bytes, n <= 0, come last).  All 32 lanes
// call it.  Whole words of 8 bytes are put together across lanes.
__device__ __forceinline__ void store_bytes_any(int8_t* p, uint2 w, int n) {
  const uint32_t t = reinterpret_cast<uintptr_t>(p) & 7;
  const int lane = threadIdx.x & 31;
  const uint64_t mine = (static_cast<uint64_t>(w.y) << 32) | w.x;
  if (t == 0) {
    if (n >= 8) {
      *reinterpret_cast<uint64_t*>(p) = mine;
    } else {
#pragma unroll 1
      for (int j = 0; j < n; ++j) p[j] = static_cast<int8_t>(mine >> (8 * j));
    }
    return;
  }
  const uint64_t before = __shfl_up_sync(0xffffffffu, mine, 1);
  int n_before = __shfl_up_sync(0xffffffffu, n, 1);
  if (lane == 0) n_before = 0;
  const int cut = 8 - static_cast<int>(t);   // bytes of a lane's own that end its first word
  if (n_before >= 8 && n >= cut) {
    *reinterpret_cast<uint64_t*>(p - t) = (before >> (8 * cut)) | (mine << (8 * t));
  } else {
#pragma unroll 1
    for (int j = cut; j < n_before && j < 8; ++j) p[j - 8] = static_cast<int8_t>(before >> (8 * j));
#pragma unroll 1
    for (int j = 0; j < n && j < cut; ++j) p[j] = static_cast<int8_t>(mine >> (8 * j));
  }
  if (lane == 31) {
#pragma unroll 1
    for (int j = cut; j < n && j < 8; ++j) p[j] = static_cast<int8_t>(mine >> (8 * j));
  }
}

// A row's scale from the encoding of its largest magnitude (of NaN where the
// row holds one: their encodings are above infinity's), and the scale's
// reciprocal.  Both are the correctly rounded f32 quotients that
// q8_quantize_per_tensor would be given and form ((float)(1.0 / (double)s)
// rounds 1 / s twice, but never to another float: s times a number of 25 bits
// has 49 at most, so 1 / s is no nearer than 2^-49 to a midpoint).  Scales
// below f32's normal numbers have no finite reciprocal: such rows count as
// zeros.  A row that holds an infinity (scale infinite, reciprocal 0) or NaN (both
// NaN) has zeros for its int8 values: 0 times such a scale is NaN, so no sum, no
// relu and no way back makes a finite number of it.
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
// encoding; see round_add_clamp_i).  Infinities and NaN give some byte, which
// TokenItem::quantize leaves out.
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

// act(g), and with GRAD act'(g) too.  F32: for f32 outputs, of exp(-|g|), which may
// be subnormal but does not overflow; silu within 3.5 units in the last place (2048
// rows, the pair 11008 x 4096 211 us, 204 by the fast ones; one row the same).  Else,
// for what is rounded to 16 bits, its exp and division are the fast ones: the sigmoid
// within (8 + 1.2 |g|) 2^-23 of itself, 2^-16 where it is furthest from 1 and still a
// normal number, a 32nd of f16's half step.  Both run into 0 or infinity where the
// sigmoid does.
template <bool GRAD, bool F32>
__device__ __forceinline__ float activate(float g, int act, float& slope) {
  if (act == kActSilu) {
    float sigma;
    if constexpr (F32) {
      const float t = expf(-fabsf(g));
      sigma = __fdiv_rn(g < 0.0f ? t : 1.0f, 1.0f + t);
    } else {
      sigma = __fdividef(1.0f, 1.0f + __expf(-g));
    }
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
// where bf16 has 8.  (Against 64 bits an f16 gradient is off by 2.9e-4 of its size, by
// 2.1e-4 with f32 operands, a bf16 one by 1.67e-3 and 1.66e-3: their own rounding is
// the rest.  A second term would double the product.)  Each row is multiplied by a
// power of two that puts a bound on its values between 2^14 and 2^15, so that f16's
// few exponents reach 29 powers of two below that bound, and the row's sums are
// divided by it again, exactly.  (Beyond 2^126 either way the row keeps what f32 can
// do.)  A bound that is no number counts as one of 2^128: it may have passed f32
// where the values do not, and those, below 2^128, then stay below 2^14; where they
// are infinite or NaN they stay so.
struct RowPower {
  float rescale, unscale;
};
__device__ __forceinline__ int exponent_bits(float v) {
  return static_cast<int>(__float_as_uint(v) >> 23) & 255;
}
// room: the power of two that the bound is put at or above, less than twice it.
// largest: of what the power multiplies on the way to the values, which it keeps
// below 2^127.
__device__ __forceinline__ RowPower row_power(float bound, int room = 14, float largest = 1.0f) {
  const int most = min(126, 253 - exponent_bits(largest));
  const int e = max(-126, min(most, 127 + room - exponent_bits(bound)));
  return {__uint_as_float(static_cast<uint32_t>(127 + e) << 23),
          __uint_as_float(static_cast<uint32_t>(127 - e) << 23)};
}
// The gated gradient's row before g and u are known: |u| and |g| are below
//   s * 127 * 128 K * (largest ws) + (largest bias)
// (of typical ones some 7 sqrt(K) times), |act| below |g|, |act'| below
// kSteepest; so with the row's largest |dh| its operand has a bound.  On the way
// to it dh times the power is multiplied by u or act(g), before a channel's scale
// makes them small: rows of almost nothing get less than f16 could take.
// tops: the gate's and the up projection's largest scale, then bias.
__device__ __forceinline__ RowPower gated_row_power(float most_dh, float s, int64_t K,
                                                    const float4& tops) {
  const float acc = fabsf(s) * (16384.0f * static_cast<float>(K));
  const float g = fmaf(acc, tops.x, tops.z), u = fmaf(acc, tops.y, tops.w);
  return row_power(most_dh * kSteepest * fmaxf(u * tops.x, g * tops.y), 14,
                   most_dh * fmaxf(1.0f, fmaxf(g, u)));
}
// Two numbers in f16, the first in the low half: one conversion.
__device__ __forceinline__ uint32_t grad_bits_x2(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// Eight values of a float row.
template <int DT>
using FloatOf = typename std::conditional<DT == Q8_F32, float, uint16_t>::type;

template <int DT, bool VEC>
struct TokenItem : RowItem<DT == Q8_F32 ? 8 : 4, VEC> {
  using RowItem<DT == Q8_F32 ? 8 : 4, VEC>::w;
  __device__ __forceinline__ void load_whole(const void* p) {   // on its boundary
#pragma unroll
    for (int j = 0; j < (DT == Q8_F32 ? 8 : 4); j += 4) {
      const uint4 v = *reinterpret_cast<const uint4*>(static_cast<const uint32_t*>(p) + j);
      w[j] = v.x;
      w[j + 1] = v.y;
      w[j + 2] = v.z;
      w[j + 3] = v.w;
    }
  }
  __device__ __forceinline__ void set(int j, FloatOf<DT> v) {
    if constexpr (DT == Q8_F32) w[j] = __float_as_uint(v);
    else w[j / 2] = (j & 1) ? (w[j / 2] & 0xffffu) | (static_cast<uint32_t>(v) << 16)
                            : (w[j / 2] & 0xffff0000u) | v;
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
    const uint32_t keep = inv > 0.0f ? 0xffffffffu : 0;   // (the same for a whole row)
    return make_uint2(four_bytes(b[0], b[1], b[2], b[3]) & keep,
                      four_bytes(b[4], b[5], b[6], b[7]) & keep);
  }
};

// Rows as items of 8 values on boundaries of 8.  VEC: rows are whole items.  Else
// a row begins t values into its first item, and what belongs to its neighbours
// counts as zeros.  (A row's values are numbered in 32 bits: K <= INT32_MAX / 2.)
template <int DT, bool VEC>
struct FlatRows {
  using T = FloatOf<DT>;
  using Item = TokenItem<DT, true>;
  struct Row {
    const T* at;
    int t, lo, hi;   // values from lo to hi lie in the matrix
  };
  const T *x, *end;
  int64_t M;
  int K, off;   // off: values that x lies behind a boundary of 8
  __device__ __forceinline__ FlatRows(const void* x_, int64_t M_, int64_t K_)
      : x(static_cast<const T*>(x_)), end(x + M_ * K_), M(M_), K(static_cast<int>(K_)),
        off(VEC ? 0 : static_cast<int>(reinterpret_cast<uintptr_t>(x_) / sizeof(T) & 7)) {}
  // Row m; past the last one, a row without values to load.
  __device__ __forceinline__ Row row(int64_t m) const {
    const T* at = x + m * K;
    Row r{at, VEC ? 0 : static_cast<int>((off + m * K) & 7), 0, m < M ? K : 0};
    if (!VEC && K >= 8) {   // (items of shorter rows reach further than one neighbour)
      if (m > 0) r.lo = -8;
      if (m + 1 < M) r.hi = K + 8;
    }
    return r;
  }
  // Item c of a row: asked for; zeros past the row.
  __device__ __forceinline__ void load(Item& it, const Row& r, int c) const {
    const int e = c * 8 - r.t;   // the row's values from e on
    it.zero();
    if constexpr (VEC) {
      if (e < r.hi) it.load_whole(r.at + e);
    } else if (e < K && r.hi > 0) {
      if (e >= r.lo && e + 8 <= r.hi) {
        it.load_whole(r.at + e);
      } else {   // the ends of the matrix
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (e + j >= 0 && e + j < K) it.set(j, r.at[e + j]);
      }
    }
  }
  // Once it is there: zeros for the neighbours' values.
  __device__ __forceinline__ void settle(Item& it, const Row& r, int c) const {
    const int e = c * 8 - r.t;
    if (!VEC && (e < 0 || e + 8 > K)) {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (e + j < 0 || e + j >= K) it.set(j, 0);
    }
  }
};

}  // namespace q8
