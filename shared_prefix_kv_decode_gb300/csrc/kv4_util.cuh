// kv4_util.cuh -- the 4-bit cache's number format: quantising K/V rows to e2m1 codes with an e4m3 scale for
// each 16 of them and a power of two for each block of tokens and head, and reading them back.
//
// With amax the largest finite magnitude of the head's elements over the block of tokens and bmax that of 16
// of them, all in exact arithmetic:
//   unit t = 2^e, e the smallest with amax <= 6 * 448 * 2^e, within [kKv4ExpMin, kKv4ExpMax];
//   scale b = the nearest e4m3 value to bmax / (6 t), at least 2^-9 and at most 448; NaN if one of the 16 is NaN;
//   code    = the nearest e2m1 value to x / (b t), saturated at +-6 (an infinity becomes +-6 b t).
// An element stands for code * b * t: 2 + 4 significant bits over a power of two, so it is exact in fp16 (without
// t), in bf16 and in fp32.  Both quotients come out as if rounded once: bmax / t and x / t are exact, and the
// correctly rounded fp32 quotient of 24 significant bits by 6 or by b (4 bits) lies on the same side of every
// halfway point (5 and 3 bits) as the exact one, or on it only together with it: numerator and halfway point
// times divisor are a unit in the last place u of the numerator apart at least, so the quotients are u / divisor,
// while half a unit of the quotient is u / 2^(k+1) at most for a divisor in [2^k, 2^(k+1)).
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cstdint>

#include "internal.h"
#include "kv8_util.cuh"

namespace granikv {

// Eight e2m1 codes (low nibble first) -> four fp16x2.
__device__ __forceinline__ void e2m1x8_to_f16x8(uint32_t w, uint32_t (&y)[4]) {
  asm("{\n .reg .b8 a, b, c, d;\n mov.b32 {a, b, c, d}, %4;\n cvt.rn.f16x2.e2m1x2 %0, a;\n cvt.rn.f16x2.e2m1x2 %1, b;\n"
      " cvt.rn.f16x2.e2m1x2 %2, c;\n cvt.rn.f16x2.e2m1x2 %3, d;\n}"
      : "=r"(y[0]), "=r"(y[1]), "=r"(y[2]), "=r"(y[3])
      : "r"(w));
}
// Eight floats -> eight e2m1 codes: nearest even, saturated at +-6.
__device__ __forceinline__ uint32_t f32x8_to_e2m1x8(const float (&x)[8]) {
  uint32_t w;
  asm("{\n .reg .b8 a, b, c, d;\n cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n"
      " cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n mov.b32 %0, {a, b, c, d};\n}"
      : "=r"(w)
      : "f"(x[0]), "f"(x[1]), "f"(x[2]), "f"(x[3]), "f"(x[4]), "f"(x[5]), "f"(x[6]), "f"(x[7]));
  return w;
}
// An e4m3 scale in both halves of an fp16x2; the product of two fp16x2 (exact: see above).
__device__ __forceinline__ uint32_t kv4_scale2(uint32_t byte) { return e4m3x2_to_f16x2((uint16_t)(byte | byte << 8)); }
__device__ __forceinline__ uint32_t f16x2_mul(uint32_t a, uint32_t b) {
  const __half2 p = __hmul2(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b));
  return *reinterpret_cast<const uint32_t*>(&p);
}
// The unit that an exponent byte stands for.
__device__ __forceinline__ float kv4_unit(uint32_t byte) { return __uint_as_float(byte << 23); }

// The exponent byte (e + 127) for a block's amax: 2688 = 1.3125 * 2^11.
__device__ __forceinline__ uint32_t kv4_exponent(float amax) {
  const uint32_t u = __float_as_uint(amax);
  const int e = (int)(u >> 23) - 11 + ((u & 0x7fffffu) > 0x280000u ? 1 : 0);
  return (uint32_t)min(max(e, 127 + kKv4ExpMin), 127 + kKv4ExpMax);
}

// 16 consecutive elements of a head.
template <typename T>
struct Kv4Group;
template <>
struct Kv4Group<__nv_bfloat16> {
  uint4 w[2];
  __device__ __forceinline__ void load(const __nv_bfloat16* src) {
    w[0] = __ldcs(reinterpret_cast<const uint4*>(src));
    w[1] = __ldcs(reinterpret_cast<const uint4*>(src) + 1);
  }
  __device__ __forceinline__ void clear() { w[0] = w[1] = make_uint4(0u, 0u, 0u, 0u); }
  // the largest magnitude as it orders among bits: above 0x7f800000 if one is NaN, 0x7f800000 if one is infinite
  __device__ __forceinline__ float top() const {
    uint32_t m = __vmaxu2(__vmaxu2(w[0].x & 0x7fff7fffu, w[0].y & 0x7fff7fffu), __vmaxu2(w[0].z & 0x7fff7fffu, w[0].w & 0x7fff7fffu));
    m = __vmaxu2(m, __vmaxu2(__vmaxu2(w[1].x & 0x7fff7fffu, w[1].y & 0x7fff7fffu), __vmaxu2(w[1].z & 0x7fff7fffu, w[1].w & 0x7fff7fffu)));
    return __uint_as_float(max(m & 0xffffu, m >> 16) << 16);
  }
  __device__ __forceinline__ float at(int i) const {
    const uint32_t u[8] = {w[0].x, w[0].y, w[0].z, w[0].w, w[1].x, w[1].y, w[1].z, w[1].w};
    return __uint_as_float(i & 1 ? u[i / 2] & 0xffff0000u : u[i / 2] << 16);
  }
};
template <>
struct Kv4Group<float> {
  float4 w[4];
  __device__ __forceinline__ void load(const float* src) {
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = __ldcs(reinterpret_cast<const float4*>(src) + i);
  }
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = make_float4(0.f, 0.f, 0.f, 0.f);
  }
  __device__ __forceinline__ float top() const {
    uint32_t m = 0u;
#pragma unroll
    for (int i = 0; i < 16; ++i) m = max(m, __float_as_uint(at(i)) & 0x7fffffffu);
    return __uint_as_float(m);
  }
  __device__ __forceinline__ float at(int i) const {
    const float4& x = w[i / 4];
    return i % 4 == 0 ? x.x : i % 4 == 1 ? x.y : i % 4 == 2 ? x.z : x.w;
  }
};
// The largest finite magnitude, given the largest.
template <typename T>
__device__ __forceinline__ float kv4_finite_top(const Kv4Group<T>& x, float top) {
  if (top < INFINITY) return top;
  float m = 0.f;
#pragma unroll
  for (int i = 0; i < 16; ++i) m = fmaxf(m, finite_abs(x.at(i)));
  return m;
}
// The group's codes and its scale's byte; top and finite: of the two functions above, byte: its block's exponent.
template <typename T>
__device__ __forceinline__ uint2 kv4_codes(const Kv4Group<T>& x, float top, float finite, uint32_t byte, uint32_t& scale) {
  const float inv_unit = kv4_unit(254u - byte);
  const uint32_t s = max((uint32_t)f32x2_to_e4m3x2(__fdiv_rn(finite * inv_unit, 6.f), 0.f), 1u);
  scale = top == top ? s : 0x7fu;
  const uint32_t f16 = e4m3x2_to_f16x2((uint16_t)s);
  const float b = __low2float(*reinterpret_cast<const __half2*>(&f16));
  // x / (b t) by one Newton step on the approximate quotient; the signs are such that a zero keeps its own
  const float minus_inv = __fdiv_rn(-1.f, b);
  uint32_t out[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    float q[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float n = x.at(8 * h + i) * -inv_unit, q0 = n * minus_inv, r = fmaf(q0, b, n);
      q[i] = r == r ? fmaf(r, minus_inv, q0) : q0;  // (an infinity stays one)
    }
    out[h] = f32x8_to_e2m1x8(q);
  }
  return make_uint2(out[0], out[1]);
}

}  // namespace granikv
