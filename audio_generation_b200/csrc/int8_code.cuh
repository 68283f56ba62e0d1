// Rounding to int8 codes, shared by the kernels that quantize.
//
// The code is the nearest integer to the exact quotient x / scale, ties to even.
// A product with the rounded reciprocal is within 2^-22 of the quotient
// relative to it, below 4e-5 in absolute terms for |quotient| <= 127.001; only
// elements within 1e-4 of a tie take the division, in 64 bits, where the
// quotient of two 32-bit floats cannot round onto a tie that it is not on (it is
// either on the tie or 2^-25 of it away).
#pragma once

#include <cuda_fp16.h>
#include <stdint.h>

#include "internal.cuh"
#include "sm100.cuh"

namespace h3 {

constexpr float kCodeMagic = 12582912.f;  // 1.5 * 2^23: adding it rounds to an integer
constexpr float kMaxFinite = 3.4028235e38f;

struct RowScale {
  float scale, inv;
  bool slow;  // the reciprocal is not a normal float: divide everywhere
};

__device__ __forceinline__ RowScale row_scale(float scale) {
  RowScale s;
  s.scale = scale;
  s.inv = 1.f / scale;
  s.slow = scale < 1e-30f;
  return s;
}

__device__ __noinline__ inline int code_by_division(float x, float factor, float scale) {
  const double q = rint((double)x * (double)factor / (double)scale);
  return (int)fmin(fmax(q, -127.0), 127.0);
}

// The low byte of the result is the code of x.
__device__ __forceinline__ uint32_t code_of(float x, const RowScale& s) {
  const float r = fmaf(x, s.inv, kCodeMagic);
  const float d = fmaf(x, s.inv, kCodeMagic - r);  // quotient - rounded quotient
  if (s.slow || fabsf(d) > 0.4999f) return (uint32_t)code_by_division(x, 1.f, s.scale);
  return __float_as_uint(r);
}

// The code of code * from under another scale (ratio = from / to): the quotient
// (code * from) / to has a 31-bit numerator, exact in 64 bits.
__device__ __forceinline__ uint32_t code_again(int code, float from, float to, float ratio) {
  const float r = fmaf((float)code, ratio, kCodeMagic);
  const float d = fmaf((float)code, ratio, kCodeMagic - r);
  if (to < 1e-30f || fabsf(d) > 0.4999f) return (uint32_t)code_by_division((float)code, from, to);
  return __float_as_uint(r);
}

// The low bytes of four words as one word.
__device__ __forceinline__ uint32_t pack4(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  return __byte_perm(__byte_perm(a, b, 0x0040), __byte_perm(c, d, 0x0040), 0x5410);
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
    if constexpr (T == H3_BF16) {
      v[2 * i] = bf16lo(w[i]);
      v[2 * i + 1] = bf16hi(w[i]);
    } else if constexpr (T == H3_F16) {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
      v[2 * i] = f.x;
      v[2 * i + 1] = f.y;
    } else {
      v[i] = __uint_as_float(w[i]);
    }
  }
}

}  // namespace h3
