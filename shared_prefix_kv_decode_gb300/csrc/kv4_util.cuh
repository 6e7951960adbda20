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
// fp32 quotient of 24 significant bits by 6 or by b (4 bits) lies on the same side of every
// halfway point (5 and 3 bits) as the exact one, or on it only together with it: numerator and halfway point
// times divisor are a unit in the last place u of the numerator apart at least, so the quotients are u / divisor,
// while half a unit of the quotient is u / 2^(k+1) at most for a divisor in [2^k, 2^(k+1)).
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cstdint>

#include "internal.h"
#include "kv8_util.cuh"
#include "tc_util.cuh"

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

// 32 bytes at once (32-byte aligned).
__device__ __forceinline__ void ldg32(const void* src, uint4& a, uint4& b) {
  asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(a.x), "=r"(a.y), "=r"(a.z), "=r"(a.w), "=r"(b.x), "=r"(b.y), "=r"(b.z), "=r"(b.w)
               : "l"(src));
}
__device__ __forceinline__ void stg32(void* dst, const uint4& a, const uint4& b) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst), "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w),
               "r"(b.x), "r"(b.y), "r"(b.z), "r"(b.w)
               : "memory");
}

// 16 consecutive elements of a head.  WIDE: from a 32-byte boundary on, else from a 16-byte one.
template <typename T>
struct Kv4Group;
template <>
struct Kv4Group<__nv_bfloat16> {
  uint4 w[2];
  template <bool WIDE>
  __device__ __forceinline__ void load(const __nv_bfloat16* src) {
    if constexpr (WIDE) {
      ldg32(src, w[0], w[1]);
    } else {
      w[0] = __ldcs(reinterpret_cast<const uint4*>(src));
      w[1] = __ldcs(reinterpret_cast<const uint4*>(src) + 1);
    }
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
  uint4 w[4];
  template <bool WIDE>
  __device__ __forceinline__ void load(const float* src) {
#pragma unroll
    for (int i = 0; i < 4; i += 2) {
      if constexpr (WIDE) {
        ldg32(src + 4 * i, w[i], w[i + 1]);
      } else {
        w[i] = __ldcs(reinterpret_cast<const uint4*>(src) + i);
        w[i + 1] = __ldcs(reinterpret_cast<const uint4*>(src) + i + 1);
      }
    }
  }
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = make_uint4(0u, 0u, 0u, 0u);
  }
  __device__ __forceinline__ float top() const {
    uint32_t m = 0u;
#pragma unroll
    for (int i = 0; i < 16; ++i) m = max(m, __float_as_uint(at(i)) & 0x7fffffffu);
    return __uint_as_float(m);
  }
  __device__ __forceinline__ float at(int i) const {
    const uint4& x = w[i / 4];
    return __uint_as_float(i % 4 == 0 ? x.x : i % 4 == 1 ? x.y : i % 4 == 2 ? x.z : x.w);
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
  // Quotients by one Newton step on n times an approximate reciprocal: exact where the true quotient is a halfway point
  // (the step's error is that of the product times that of the reciprocal, 2^-44 of it), and elsewhere within half a
  // unit in the last place and that, which is on the true one's side.
  const float inv_unit = kv4_unit(254u - byte);
  const float n6 = finite * inv_unit, q6 = n6 * (1.f / 6.f);
  const uint32_t s = max((uint32_t)f32x2_to_e4m3x2(fmaf(fmaf(-q6, 6.f, n6), 1.f / 6.f, q6), 0.f), 1u);
  scale = top == top ? s : 0x7fu;
  const uint32_t f16 = e4m3x2_to_f16x2((uint16_t)s);
  const float b = __low2float(*reinterpret_cast<const __half2*>(&f16));
  float minus_inv;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(minus_inv) : "f"(-b));
  // (the signs are such that a zero keeps its own)
  const uint64_t f2 = f2_pack(-inv_unit, -inv_unit), i2 = f2_pack(minus_inv, minus_inv), b2 = f2_pack(b, b);
  const bool plain = top < INFINITY;
  uint32_t out[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    float q[8];
    if (plain) {
#pragma unroll
      for (int i = 0; i < 8; i += 2) {
        const uint64_t n = f2_mul(f2_pack(x.at(8 * h + i), x.at(8 * h + i + 1)), f2), q0 = f2_mul(n, i2);
        f2_unpack(f2_fma(f2_fma(q0, b2, n), i2, q0), q[i], q[i + 1]);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float n = x.at(8 * h + i) * -inv_unit, q0 = n * minus_inv, r = fmaf(q0, b, n);
        q[i] = r == r ? fmaf(r, minus_inv, q0) : q0;  // (an infinity stays one)
      }
    }
    out[h] = f32x8_to_e2m1x8(q);
  }
  return make_uint2(out[0], out[1]);
}

}  // namespace granikv
