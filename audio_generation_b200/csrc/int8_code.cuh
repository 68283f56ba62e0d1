// Rounding to int8 codes, shared by the kernels that quantize.
//
// The code is the nearest integer to the exact quotient x / scale, ties to even.
// x times the correctly rounded reciprocal is within 2^-24 of the quotient
// relative to it, so its floor r is the quotient's or, next to an integer, that
// integer's neighbour; either way the code is r or r + 1. The rest x - r scale
// decides: r + 1 if it is more than half the scale, or equal to that and r odd.
// One fused multiply-add gives the rest exactly wherever the decision is close: it
// is a multiple of the scale's last place and at most about the scale (for x
// below the scale it is x itself, or the scale less |x|, which is exact from half
// the scale on; where it is rounded, r is -1 and half the scale counts as more).
// (Near-ties are not rare: with x and the maximum in bfloat16 the quotient is 127
// times a ratio of two 8-bit numbers.)
#pragma once

#include <cuda_fp16.h>
#include <stdint.h>

#include "internal.cuh"
#include "sm100.cuh"
#include "softmax.cuh"

namespace h3 {

constexpr float kCodeMagic = 12582912.f;  // 1.5 * 2^23: adding it leaves an integer
constexpr float kMaxFinite = 3.4028235e38f;

struct RowScale {
  float scale, inv;
  float up, limit;  // a power of two times the scale's exponent: see codes_of
  bool slow;        // too small for exact rests: divide everywhere, in 64 bits
  bool ties;        // an element of the row's type can lie on a tie
};

// For elements of type T. x on a tie means 2 x = (2 r + 1) scale exactly, so the
// scale's mantissa without its trailing zeros has no more bits than x's: 8 in
// bfloat16, 11 in fp16; a scale that is a rounded quotient hardly ever does.
template <h3_type T>
__device__ __forceinline__ RowScale row_scale(float scale) {
  RowScale s;
  const uint32_t bits = __float_as_uint(scale);
  s.scale = scale;
  s.inv = 1.f / scale;
  s.slow = scale < 1e-30f;
  s.up = __uint_as_float((280u - (bits >> 23)) << 23);  // 2^26 over the scale's power of two
  s.limit = -0.5f * scale * s.up;
  s.ties = T == H3_F32 || (bits & (T == H3_BF16 ? 0xffffu : 0x1fffu)) == 0;
  return s;
}

__device__ __noinline__ inline int code_by_division(float x, float factor, float scale) {
  const double q = rint((double)x * (double)factor / (double)scale);
  return (int)fmin(fmax(q, -127.0), 127.0);
}

// Eight codes by division, one call for all: the rare way.
__device__ __noinline__ inline uint2 codes8_by_division(float a, float b, float c, float d, float e,
                                                        float f, float g, float h, float scale) {
  uint32_t w[2] = {0, 0};
  const float x[8] = {a, b, c, d, e, f, g, h};
#pragma unroll
  for (int i = 0; i < 8; ++i)
    w[i / 4] |= ((uint32_t)code_by_division(x[i], 1.f, scale) & 0xffu) << (8 * (i & 3));
  return make_uint2(w[0], w[1]);
}

// The low bytes of four words as one word.
__device__ __forceinline__ uint32_t pack4(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  return __byte_perm(__byte_perm(a, b, 0x0040), __byte_perm(c, d, 0x0040), 0x5410);
}

// N floors (as kCodeMagic + floor) and their rests; two elements per instruction.
template <int N>
__device__ __forceinline__ void floors(const float* x, float scale, float inv, float* r,
                                       float* rest) {
  const uint64_t inv2 = f2_pack(inv, inv), magic = f2_pack(kCodeMagic, kCodeMagic);
  const uint64_t unmagic = f2_pack(-kCodeMagic, -kCodeMagic), minus = f2_pack(-scale, -scale);
#pragma unroll
  for (int i = 0; i < N; i += 2) {
    const uint64_t v = f2_pack(x[i], x[i + 1]);
    const uint64_t rr = f2_fma_down(v, inv2, magic);
    f2_unpack(f2_fma(f2_add(rr, unmagic), minus, v), rest[i], rest[i + 1]);
    f2_unpack(rr, r[i], r[i + 1]);
  }
}

template <int N>
__device__ __forceinline__ uint2 pack_codes(const uint32_t* u) {
  return make_uint2(pack4(u[0], u[1], u[2], u[3]),
                    N == 8 ? pack4(u[N - 4], u[N - 3], u[N - 2], u[N - 1]) : 0);
}

// The codes of N = 8 or 4 elements (.y is then void), ties decided too.
template <int N>
__device__ __forceinline__ uint2 codes_with_ties(const float* x, float scale, float inv) {
  float r[N], rest[N];
  floors<N>(x, scale, inv, r, rest);
  const uint32_t half = __float_as_uint(0.5f * scale);
  uint32_t u[N];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const uint32_t w = __float_as_uint(r[i]);
    // above half the scale, or from half the scale on where r is odd
    u[i] = w + (rest[i] > __uint_as_float(half - (w & 1u)) ? 1u : 0u);
  }
  return pack_codes<N>(u);
}

// Out of line: few rows of 16-bit elements come here.
__device__ __noinline__ inline uint2 codes8_careful(float a, float b, float c, float d, float e,
                                                    float f, float g, float h, float scale,
                                                    float inv, bool slow) {
  if (slow) return codes8_by_division(a, b, c, d, e, f, g, h, scale);
  const float x[8] = {a, b, c, d, e, f, g, h};
  return codes_with_ties<8>(x, scale, inv);
}

// The codes of x[0..7] of a 16-bit type.
__device__ __forceinline__ uint2 codes_of_8(const float* x, const RowScale& s) {
  if (s.slow || s.ties)
    return codes8_careful(x[0], x[1], x[2], x[3], x[4], x[5], x[6], x[7], s.scale, s.inv, s.slow);
  float r[8], rest[8];
  floors<8>(x, s.scale, s.inv, r, rest);
  // (rest - scale / 2) times a power of two is at least 4 or below 0: limited to
  // [0, 1] it is what r lacks. (On the FMA pipe; compares and selects run at half
  // its rate, and the kernels' time goes to them: 62 -> 55 us for 8192 x 14336.)
  uint32_t u[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) u[i] = __float_as_uint(r[i] + fma_01(rest[i], s.up, s.limit));
  return pack_codes<8>(u);
}

// The codes of x[0..3] of float32.
__device__ __forceinline__ uint32_t codes_of_4(const float* x, const RowScale& s) {
  if (s.slow) return codes8_by_division(x[0], x[1], x[2], x[3], 0, 0, 0, 0, s.scale).x;
  return codes_with_ties<4>(x, s.scale, s.inv).x;
}

// The code of code * from under another scale (ratio = from / to, within 2^-22):
// the quotient (code * from) / to has a 31-bit numerator, exact in 64 bits.
__device__ __forceinline__ uint32_t code_again(int code, float from, float to, float ratio) {
  const float r = fmaf((float)code, ratio, kCodeMagic);
  const float d = fmaf((float)code, ratio, kCodeMagic - r);
  if (to < 1e-30f || fabsf(d) > 0.4999f) return (uint32_t)code_by_division((float)code, from, to);
  return __float_as_uint(r);
}

// Two neighbouring 16-bit elements as floats.
template <h3_type T>
__device__ __forceinline__ void unpack_pair(uint32_t w, float& lo, float& hi) {
  if constexpr (T == H3_BF16) {
    lo = bf16lo(w);
    hi = bf16hi(w);
  } else {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w));
    lo = f.x;
    hi = f.y;
  }
}

// 16 bytes of a row as floats: 8 elements of 2 bytes, or 4 of 4.
template <h3_type T>
struct Vec {
  static constexpr int N = T == H3_F32 ? 4 : 8;
};
template <h3_type T>
__device__ __forceinline__ void unpack(const uint4& u, float* v) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (T == H3_F32) v[i] = __uint_as_float(w[i]);
    else unpack_pair<T>(w[i], v[2 * i], v[2 * i + 1]);
  }
}

// The warp's largest magnitude, a NaN winning: the bits of floats >= 0 and of
// positive NaNs are ordered as integers are (one instruction for the warp).
__device__ __forceinline__ float warp_peak(float m) {
  return __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(m) & 0x7fffffffu));
}

// max(m, |elements|) of 16 bytes of a row, a NaN winning: 16-bit types by pairs in
// their own type, where maxima are exact (m with any sign until its value is taken).
template <h3_type T>
struct AbsMax;
template <>
struct AbsMax<H3_F32> {
  float m = 0.f;
  __device__ __forceinline__ void add(const uint4& u) {
    m = max_nan(m, fabsf(__uint_as_float(u.x)));
    m = max_nan(m, fabsf(__uint_as_float(u.y)));
    m = max_nan(m, fabsf(__uint_as_float(u.z)));
    m = max_nan(m, fabsf(__uint_as_float(u.w)));
  }
  __device__ __forceinline__ float value() const { return m; }
};
template <>
struct AbsMax<H3_BF16> {
  uint32_t m = 0;
  __device__ __forceinline__ void one(uint32_t w) {
    asm("max.NaN.xorsign.abs.bf16x2 %0, %0, %1;" : "+r"(m) : "r"(w));
  }
  __device__ __forceinline__ void add(const uint4& u) { one(u.x), one(u.y), one(u.z), one(u.w); }
  __device__ __forceinline__ float value() const {
    return max_nan(fabsf(bf16lo(m)), fabsf(bf16hi(m)));
  }
};
template <>
struct AbsMax<H3_F16> {
  uint32_t m = 0;
  __device__ __forceinline__ void one(uint32_t w) {
    asm("max.NaN.xorsign.abs.f16x2 %0, %0, %1;" : "+r"(m) : "r"(w));
  }
  __device__ __forceinline__ void add(const uint4& u) { one(u.x), one(u.y), one(u.z), one(u.w); }
  __device__ __forceinline__ float value() const {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&m));
    return max_nan(fabsf(f.x), fabsf(f.y));
  }
};

}  // namespace h3
