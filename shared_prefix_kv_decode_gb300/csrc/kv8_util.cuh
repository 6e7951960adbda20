// kv8_util.cuh -- the 8-bit cache's number format: quantising K/V rows to e4m3 codes, and reading
// codes back.  Every e4m3 value is exact in fp16 (4 significant bits, exponents -9..8), so the
// attention kernels convert codes to fp16 with one hardware conversion per pair and apply the
// scales to the scores and weights in fp32.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cstdint>

#include "internal.h"

namespace granikv {

// Two e4m3 codes (low byte first) -> fp16x2.
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint16_t w) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(w));
  return r;
}
// Four e4m3 codes -> two fp16x2 (codes 0, 1 and 2, 3).
__device__ __forceinline__ void e4m3x4_to_f16x4(uint32_t w, uint32_t& lo, uint32_t& hi) {
  asm("{\n .reg .b16 l, h;\n mov.b32 {l, h}, %2;\n cvt.rn.f16x2.e4m3x2 %0, l;\n cvt.rn.f16x2.e4m3x2 %1, h;\n}"
      : "=r"(lo), "=r"(hi)
      : "r"(w));
}
__device__ __forceinline__ void e4m3x4_to_f32x4(uint32_t w, float (&x)[4]) {
  uint32_t a, b;
  e4m3x4_to_f16x4(w, a, b);
  const float2 u = __half22float2(*reinterpret_cast<__half2*>(&a)), v = __half22float2(*reinterpret_cast<__half2*>(&b));
  x[0] = u.x;
  x[1] = u.y;
  x[2] = v.x;
  x[3] = v.y;
}
// Two floats -> two e4m3 codes (a in the low byte): nearest even, saturated at +-448, NaN kept.
__device__ __forceinline__ uint16_t f32x2_to_e4m3x2(float a, float b) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(b), "f"(a));
  return r;
}
__device__ __forceinline__ uint32_t f32x4_to_e4m3x4(float a, float b, float c, float d) {
  return (uint32_t)f32x2_to_e4m3x2(a, b) | ((uint32_t)f32x2_to_e4m3x2(c, d) << 16);
}

// Products of two pairs of floats.
__device__ __forceinline__ uint64_t f2_mul(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

// A query row scaled by a power of two so that its largest finite element lies in [2^kTop, 2^(kTop+1)).
// In fp16 with kTop = 14: bf16's 8 significant bits fit fp16's 11, so elements down to 2^-31 of the largest stay
// exact (fp16's last subnormal is 2^-24), smaller ones are off by at most 2^-39 of it.
__device__ __forceinline__ float bf16x2_finite_max(uint32_t w) {
  const float a = fabsf(__uint_as_float(w << 16)), b = fabsf(__uint_as_float(w & 0xffff0000u));
  return fmaxf(a < INFINITY ? a : 0.f, b < INFINITY ? b : 0.f);
}
// The power of two for a row whose largest finite element is amax, and the one that undoes it; both
// are kept within what fp32 holds.
template <int kTop>
__device__ __forceinline__ float q_factor(float amax, float& unit) {
  const int e = (int)((__float_as_uint(amax) >> 23) & 255u);
  const int up = amax == 0.f ? 127 : min(kTop + 127 + 127 - e, 253);  // 2^(kTop - exponent of amax)
  unit = __uint_as_float((uint32_t)(254 - up) << 23);
  return __uint_as_float((uint32_t)up << 23);
}
__device__ __forceinline__ uint32_t bf16x2_to_f16x2(uint32_t w, float f) {
  const __half2 h = __floats2half2_rn(__uint_as_float(w << 16) * f, __uint_as_float(w & 0xffff0000u) * f);
  return *reinterpret_cast<const uint32_t*>(&h);
}
// The same for a row spread over the four lanes of a quad, W words of two bf16 a lane.
template <int W>
__device__ __forceinline__ void q_to_f16(uint32_t* w, float& unit) {
  float amax = 0.f;
#pragma unroll
  for (int i = 0; i < W; ++i) amax = fmaxf(amax, bf16x2_finite_max(w[i]));
  amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
  amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
  const float f = q_factor<14>(amax, unit);
#pragma unroll
  for (int i = 0; i < W; ++i) w[i] = bf16x2_to_f16x2(w[i], f);
}
// q as the attention kernels take it: an infinity becomes NaN (0 * inf; a NaN stays one, 0 * x + x is any other x).
// The scores of an infinity may all be -inf, which looks like a row without keys.
__device__ __forceinline__ float q_no_inf(float x) { return fmaf(0.f, x, x); }
__device__ __forceinline__ __half2 q_no_inf(__half2 x) { return __hfma2(__floats2half2_rn(0.f, 0.f), x, x); }

// A partial row's log-sum-exp as the merge takes it: -inf for a row without weight, +inf for one whose
// weights hold a NaN (the merge's maximum passes over a NaN; +inf makes the whole row NaN).
__device__ __forceinline__ float kv8_record_lse(float sum, float lse) {
  return sum == 0.f ? -INFINITY : sum == sum ? lse : INFINITY;
}

// |x| for a block's amax: infinities and NaN do not count.
__device__ __forceinline__ float finite_abs(float x) {
  const float a = fabsf(x);
  return a < INFINITY ? a : 0.f;
}
__device__ __forceinline__ float kv8_scale(float amax) { return fmaxf(amax, kKv8AmaxMin) / kE4m3Max; }

// x * 448 / amax, such that its conversion to e4m3 is the nearest code of the exact quotient: with a the
// significand of amax and f = 448 over its power of two (exact), the quotient of x f and a.  One
// Newton step on the approximate quotient makes it the correctly rounded one of what it divides.
// bf16: x f is exact (8 + 3 bits), and the exact quotient is either halfway between two codes, then it is
// q itself, or 2^-13 or more away from that.
// fp32: x f takes 27 bits, in two parts; the exact quotient may lie closer to a halfway point than
// fp32 resolves, so q is rounded to odd: of the two neighbours of a quotient that fp32 does not hold, the
// one with an odd last bit, which lies on its side of every halfway point.
// An x that is not finite gives itself.
// (The signs are such that the last sum keeps that of a zero.)
struct Kv8Divisor {
  float minus_f, a, minus_inv;
};
__device__ __forceinline__ Kv8Divisor kv8_divisor(float amax) {
  const uint32_t u = __float_as_uint(fmaxf(amax, kKv8AmaxMin));
  const float a = __uint_as_float((u & 0x7fffffu) | 0x3f800000u);
  return {-__uint_as_float(((262u - (u >> 23)) << 23) | 0x600000u), a, -1.f / a};  // 1.75 * 2^(8 - exponent)
}
template <typename T>
__device__ __forceinline__ float kv8_quotient(float x, const Kv8Divisor& by);
template <>
__device__ __forceinline__ float kv8_quotient<__nv_bfloat16>(float x, const Kv8Divisor& by) {
  const float n = x * by.minus_f, q0 = n * by.minus_inv, r = fmaf(q0, by.a, n);
  return r == r ? fmaf(r, by.minus_inv, q0) : x;
}
template <>
__device__ __forceinline__ float kv8_quotient<float>(float x, const Kv8Divisor& by) {
  const float n = x * by.minus_f, low = fmaf(x, by.minus_f, -n), q0 = n * by.minus_inv;
  const float r = fmaf(q0, by.a, n) + low;
  if (!(r == r)) return x;
  const float q = fmaf(r, by.minus_inv, q0), over = fmaf(q, by.a, n) + low;  // q a - x f
  uint32_t u = __float_as_uint(q);
  if (over != 0.f && q != 0.f && !(u & 1u)) u = (over < 0.f) == (q > 0.f) ? u + 1u : u - 1u;
  return __uint_as_float(u);
}

}  // namespace granikv
