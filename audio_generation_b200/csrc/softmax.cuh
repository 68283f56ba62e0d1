// Arithmetic shared by the attention kernels' softmax: the MUFU exponential,
// packed fp32 pairs, an exponential on the FMA pipe, a three-way maximum and one
// that keeps NaN.
#pragma once

#include <stdint.h>

namespace h3 {

__device__ __forceinline__ float exp2_mufu(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Packed fp32 pair arithmetic (one instruction for two lanes of work).
__device__ __forceinline__ uint64_t f2_pack(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ void f2_unpack(uint64_t v, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ uint64_t f2_fma(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t f2_fma_down(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;  // rounded towards minus infinity
  asm("fma.rm.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t f2_mul(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint64_t f2_add(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

// 2^x for two values on the FMA pipe: x = j + f with j = round(x) (by adding
// `magic` = 1.5 * 2^23, which leaves the integer in the low mantissa bits) and f
// in [-1/2, 1/2], 2^f by a cubic, j added to the exponent. Inputs are at least -126,
// or -127 where the cubic is 1 at 0 (0 then comes out).
struct Cubic {
  float c3, c2, c1, c0, magic;
};
__device__ __forceinline__ void exp2_cubic2_clamped(uint64_t xc, const Cubic& c, float& p0,
                                                    float& p1) {
  const uint64_t t = f2_add(xc, f2_pack(c.magic, c.magic));
  const uint64_t jf = f2_add(t, f2_pack(-c.magic, -c.magic));  // j, exact
  const uint64_t f = f2_fma(jf, f2_pack(-1.f, -1.f), xc);      // x - j, exact
  uint64_t p = f2_fma(f2_pack(c.c3, c.c3), f, f2_pack(c.c2, c.c2));
  p = f2_fma(p, f, f2_pack(c.c1, c.c1));
  p = f2_fma(p, f, f2_pack(c.c0, c.c0));
  float q0, q1, t0, t1;
  f2_unpack(p, q0, q1);
  f2_unpack(t, t0, t1);
  p0 = __int_as_float(__float_as_int(q0) + (__float_as_int(t0) << 23));
  p1 = __int_as_float(__float_as_int(q1) + (__float_as_int(t1) << 23));
}
__device__ __forceinline__ void exp2_cubic2(uint64_t x2, const Cubic& c, float& p0, float& p1) {
  float x0, x1;
  f2_unpack(x2, x0, x1);
  exp2_cubic2_clamped(f2_pack(fmaxf(x0, -126.f), fmaxf(x1, -126.f)), c, p0, p1);
}

__device__ __forceinline__ float fma_01(float a, float b, float c) {  // limited to [0, 1]
  float d;
  asm("fma.rn.sat.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

__device__ __forceinline__ float max_nan(float a, float b) {  // a NaN wins
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

}  // namespace h3
