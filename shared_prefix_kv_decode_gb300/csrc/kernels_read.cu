// kernels_read.cu -- rows of a pool back as [N, n_kv, d]: of a 16- or 32-bit pool as they are, of a packed one as
// the values that its codes and scales stand for, rounded once.
// 4 bits: exact in bf16 and fp32.  8 bits: code times scale in fp32, then to the type, which for bf16 gives what one
// rounding of the product gives.  A block's scale is a / 448 = a / 7 / 64 with a of 8 significant bits (rounded by 2^-24).  With c the
// code's 4 bits, c a / 7 differs from a point halfway between two bf16 values (9 bits) by 1 / (2 c a) >= 2^-13 of itself at
// least, far more than fp32 rounds; or equals it, only if 7 divides a (a point of 9 bits is not 1 or 2 times a), and
// then scale and product are exact.
#include "kv4_util.cuh"
#include "launch_util.cuh"
#include "tc_util.cuh"

#include <type_traits>

namespace granikv {
namespace {

// WIDE: to a 32-byte boundary, else to a 16-byte one.  In one store, a warp's stores fill whole sectors: 16K tokens of
// 8 x 128 in 4 bits take 15.5 us, 0.82 of the copy rate.
template <bool WIDE>
__device__ __forceinline__ void store32(void* dst, const uint4& a, const uint4& b) {
  if constexpr (WIDE) {
    stg32(dst, a, b);
  } else {
    reinterpret_cast<uint4*>(dst)[0] = a;
    reinterpret_cast<uint4*>(dst)[1] = b;
  }
}
template <bool WIDE>
__device__ __forceinline__ void store16(__nv_bfloat16* dst, const float (&x)[16]) {
  uint32_t w[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const __nv_bfloat162 p = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&p);
  }
  store32<WIDE>(dst, make_uint4(w[0], w[1], w[2], w[3]), make_uint4(w[4], w[5], w[6], w[7]));
}
template <bool WIDE>
__device__ __forceinline__ void store16(float* dst, const float (&x)[16]) {
#pragma unroll
  for (int i = 0; i < 16; i += 8)
    store32<WIDE>(dst + i, *reinterpret_cast<const uint4*>(x + i), *reinterpret_cast<const uint4*>(x + i + 4));
}

constexpr int kDeep = 4;  // (16K tokens of 8 x 128 in 4 bits: one piece a thread 16.4 us, two 15.5, four 15.5, eight 16.1)

// 16 elements of one head of a row, as they stand there.
template <int BITS, typename T>
struct Held {
  static constexpr int kWords = BITS == 0 ? 16 * sizeof(T) / 16 : 1;
  uint4 w[kWords];   // 4 bits: .x and .y codes
  uint32_t scale, unit;
  __device__ __forceinline__ void load(const uint8_t* __restrict__ row, int32_t n_kv, int32_t d, int32_t j, int32_t piece) {
    if constexpr (BITS == 0) {
      const uint4* src = reinterpret_cast<const uint4*>(row) + ((int64_t)j * (d / 16) + piece) * kWords;
#pragma unroll
      for (int i = 0; i < kWords; ++i) w[i] = __ldcs(src + i);
    } else if constexpr (BITS == 8) {
      w[0] = __ldcs(reinterpret_cast<const uint4*>(row + (int64_t)j * d + piece * 16));
      scale = *reinterpret_cast<const uint32_t*>(row + (int64_t)n_kv * d + 4 * j);
    } else {
      const uint2 x = __ldcs(reinterpret_cast<const uint2*>(row + (int64_t)j * (d / 2) + piece * 8));
      w[0] = make_uint4(x.x, x.y, 0u, 0u);
      scale = row[kv4_scales_at(n_kv, d) + (int64_t)j * (d / kKv4Group) + piece];
      unit = row[kv4_units_at(n_kv, d) + j];
    }
  }
  template <bool WIDE>
  __device__ __forceinline__ void store(T* __restrict__ dst) const {
    if constexpr (BITS == 0) {
#pragma unroll
      for (int i = 0; i < kWords; i += 2) store32<WIDE>(reinterpret_cast<uint4*>(dst) + i, w[i], w[i + 1]);
      return;
    }
    float x[16];
    if constexpr (BITS == 8) {
      const uint32_t u[4] = {w[0].x, w[0].y, w[0].z, w[0].w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float f[4];
        e4m3x4_to_f32x4(u[i], f);
#pragma unroll
        for (int c = 0; c < 4; ++c) x[4 * i + c] = f[c] * __uint_as_float(scale);
      }
    } else {
      const uint32_t b = kv4_scale2(scale);
      const float t = kv4_unit(unit);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t y[4];
        e2m1x8_to_f16x8(h ? w[0].y : w[0].x, y);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t p = f16x2_mul(y[i], b);
          const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&p));
          x[8 * h + 2 * i] = f.x * t;
          x[8 * h + 2 * i + 1] = f.y * t;
        }
      }
    }
    store16<WIDE>(dst, x);
  }
};

// A thread takes DEEP pieces of 16 elements of the CTA's tokens, all of them requested before the first is stored.
template <int BITS, typename T, bool WIDE, int DEEP>
__global__ void __launch_bounds__(256) read_kernel(ReadParams p, int32_t d, int32_t tokens) {
  const int32_t per_head = d / 16, per_row = p.n_kv * per_head;
  const uint8_t* pool = blockIdx.y ? p.pool[1] : p.pool[0];
  T* out = (T*)(blockIdx.y ? p.out[1] : p.out[0]);
  const int64_t t0 = (int64_t)blockIdx.x * tokens;
  const int32_t n = (int32_t)min((int64_t)tokens, p.N - t0) * per_row;
  for (int32_t i0 = threadIdx.x; i0 < n; i0 += 256 * DEEP) {
    Held<BITS, T> x[DEEP];
    bool have[DEEP];
#pragma unroll
    for (int k = 0; k < DEEP; ++k) {
      const int32_t i = i0 + 256 * k, t = i / per_row, h = i - t * per_row, j = h / per_head;
      have[k] = i < n;
      if (!have[k]) continue;
      int64_t slot = p.first_slot + t0 + t;
      if (p.slots) {
        slot = p.slots[t0 + t];
        if (slot < p.n_hot || slot >= p.n_slots) {  // its row is left as it was
          if (h == 0) atomicCAS(p.err, 0, (int32_t)kDevBadSlot);
          have[k] = false;
          continue;
        }
      }
      x[k].load(pool + slot * p.row, p.n_kv, d, j, h - j * per_head);
    }
#pragma unroll
    for (int k = 0; k < DEEP; ++k)
      if (have[k]) x[k].template store<WIDE>(out + (t0 * per_row + i0 + 256 * k) * 16);
  }
}

template <int BITS, typename T>
cudaError_t read_bits(int32_t d, const ReadParams& p, cudaStream_t s) {
  // kDeep pieces a thread; one, where the CTAs are too few to fill the SMs.
  const int64_t per_row = (int64_t)p.n_kv * (d / 16);
  if (per_row > INT32_MAX / 2) return cudaErrorInvalidValue;
  const bool deep = p.N * per_row >= 512 * 1024;
  const int64_t pieces = deep ? 256 * kDeep : 256;
  const int32_t tokens = (int32_t)(per_row >= pieces ? 1 : pieces / per_row);
  const dim3 grid((unsigned)(((int64_t)p.N + tokens - 1) / tokens), 2);
  const bool wide = ((uintptr_t)p.out[0] | (uintptr_t)p.out[1]) % 32 == 0;
  auto kernel = !wide ? read_kernel<BITS, T, false, 1> : deep ? read_kernel<BITS, T, true, kDeep> : read_kernel<BITS, T, true, 1>;
  kernel<<<grid, 256, 0, s>>>(p, d, tokens);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_read(int32_t dtype, int32_t bits, int32_t d, const ReadParams& p, cudaStream_t s) {
  auto of = [&](auto t) {
    using T = decltype(t);
    return bits == 8 ? read_bits<8, T>(d, p, s) : bits == 4 ? read_bits<4, T>(d, p, s) : read_bits<0, T>(d, p, s);
  };
  return dtype == 1 ? of(__nv_bfloat16{}) : of(0.f);
}

}  // namespace granikv
