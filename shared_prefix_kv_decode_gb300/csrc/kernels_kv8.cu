// kernels_kv8.cu -- 8-bit cache: the kernels that quantise K/V rows into packed slots, and the launch of
// the CUDA-core decode attention over such slots (packed_generic_body.cuh).
#include "kv8_util.cuh"
#include "launch_util.cuh"
#include "packed_generic_body.cuh"
#include "tc_util.cuh"

#include <cmath>

namespace granikv {
namespace {

// 16 bytes of a row, kept as they came: 8 bf16 or 4 fp32 elements.  amax_of: the largest finite magnitude
// of N pieces.
template <typename T>
struct Piece;
template <>
struct Piece<__nv_bfloat16> {
  static constexpr int kElems = 8;
  uint4 w;
  // (kv8_quotient, two elements to an instruction)
  __device__ __forceinline__ void store(uint8_t* dst, const Kv8Divisor& by, bool finite) const {
    const uint64_t f2 = f2_pack(by.minus_f, by.minus_f), inv2 = f2_pack(by.minus_inv, by.minus_inv), a2 = f2_pack(by.a, by.a);
    auto codes = [&](uint32_t w) {
      const float x = __uint_as_float(w << 16), y = __uint_as_float(w & 0xffff0000u);
      float a, b;
      if (finite) {
        const uint64_t n = f2_mul(f2_pack(x, y), f2), q0 = f2_mul(n, inv2), r = f2_fma(q0, a2, n);
        f2_unpack(f2_fma(r, inv2, q0), a, b);
      } else {
        a = kv8_quotient<__nv_bfloat16>(x, by);
        b = kv8_quotient<__nv_bfloat16>(y, by);
      }
      return (uint32_t)f32x2_to_e4m3x2(a, b);
    };
    *reinterpret_cast<uint2*>(dst) = make_uint2(codes(w.x) | codes(w.y) << 16, codes(w.z) | codes(w.w) << 16);
  }
  template <int N>
  __device__ static __forceinline__ float amax_of(const Piece (&x)[N], bool& finite) {
    // magnitudes order as their bits do, two to a word; only where one is not finite are they told apart
    uint32_t m = 0u;
#pragma unroll
    for (int c = 0; c < N; ++c) {
      m = __vmaxu2(m, __vmaxu2(x[c].w.x & 0x7fff7fffu, x[c].w.y & 0x7fff7fffu));
      m = __vmaxu2(m, __vmaxu2(x[c].w.z & 0x7fff7fffu, x[c].w.w & 0x7fff7fffu));
    }
    const uint32_t top = max(m & 0xffffu, m >> 16);
    float amax = __uint_as_float(top << 16);
    finite = top < 0x7f80u;
    if (!finite) {
      amax = 0.f;
#pragma unroll
      for (int c = 0; c < N; ++c)
        amax = fmaxf(amax, fmaxf(fmaxf(bf16x2_finite_max(x[c].w.x), bf16x2_finite_max(x[c].w.y)),
                                 fmaxf(bf16x2_finite_max(x[c].w.z), bf16x2_finite_max(x[c].w.w))));
    }
    return amax;
  }
};
template <>
struct Piece<float> {
  static constexpr int kElems = 4;
  uint4 w;
  __device__ __forceinline__ void store(uint8_t* dst, const Kv8Divisor& by, bool) const {
    auto q = [&](uint32_t u) { return kv8_quotient<float>(__uint_as_float(u), by); };
    *reinterpret_cast<uint32_t*>(dst) = f32x4_to_e4m3x4(q(w.x), q(w.y), q(w.z), q(w.w));
  }
  template <int N>
  __device__ static __forceinline__ float amax_of(const Piece (&x)[N], bool&) {
    float amax = 0.f;
#pragma unroll
    for (int c = 0; c < N; ++c)
      amax = fmaxf(amax, fmaxf(fmaxf(finite_abs(__uint_as_float(x[c].w.x)), finite_abs(__uint_as_float(x[c].w.y))),
                               fmaxf(finite_abs(__uint_as_float(x[c].w.z)), finite_abs(__uint_as_float(x[c].w.w)))));
    return amax;
  }
};

// One block of kPackedBlock slab tokens of one KV head (the heads of a block are neighbours in the grid, so
// that its rows are read and written whole at about the same time), of K (blockIdx.y = 0) or V.  The block stays in
// registers between its amax and its codes (pieces of 16 bytes, all of a thread's requested at once), so
// the rows are read once: 3 bytes moved for each bf16 element (16K tokens of 8 x 128: 18.7 us at six CTAs an
// SM; its 100 MB take 14.9).  What it costs beyond HBM is issue: 17.4 us with one product an element in place of
// the quotient (which rounds twice), 23.2 with head_dim at run time (two divisions for each piece's place).
template <typename T, int D>
__global__ void __launch_bounds__(256, sizeof(T) * D <= 256 ? 6 : 1) kv8_fill_kernel(
    const T* __restrict__ k, const T* __restrict__ v, int32_t L_p, uint8_t* __restrict__ kpool,
    uint8_t* __restrict__ vpool, int64_t first_slot, int32_t n_kv) {
  constexpr int kElems = Piece<T>::kElems;
  constexpr int kPerRow = D / kElems;              // pieces of a head's row
  constexpr int kPieces = kPackedBlock * kPerRow / 256;  // of a thread
  __shared__ float s_max[8];
  const int32_t j = blockIdx.x % n_kv;
  const int32_t t0 = blockIdx.x / n_kv * kPackedBlock;
  const int32_t n = min(kPackedBlock, L_p - t0);
  const T* src = (blockIdx.y ? v : k) + ((int64_t)t0 * n_kv + j) * D;
  Piece<T> x[kPieces];
#pragma unroll
  for (int c = 0; c < kPieces; ++c) {
    const int32_t idx = threadIdx.x + c * 256, t = idx / kPerRow;
    x[c].w = t < n ? __ldcs(reinterpret_cast<const uint4*>(src + t * (n_kv * D) + idx % kPerRow * kElems))
                   : make_uint4(0u, 0u, 0u, 0u);
  }
  bool finite = true;  // this thread's elements
  float amax = Piece<T>::amax_of(x, finite);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
  if ((threadIdx.x & 31) == 0) s_max[threadIdx.x >> 5] = amax;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < 8; ++w) amax = fmaxf(amax, s_max[w]);
  const Kv8Divisor by = kv8_divisor(amax);
  const float scale = kv8_scale(amax);
  const int32_t row = (int32_t)kv8_row_bytes(n_kv, D);
  uint8_t* dst = (blockIdx.y ? vpool : kpool) + (first_slot + t0) * row;
#pragma unroll
  for (int c = 0; c < kPieces; ++c) {
    const int32_t idx = threadIdx.x + c * 256, t = idx / kPerRow;
    if (t < n) x[c].store(dst + t * row + j * D + idx % kPerRow * kElems, by, finite);
  }
  for (int32_t t = threadIdx.x; t < n; t += 256) *reinterpret_cast<float*>(dst + t * row + n_kv * D + 4 * j) = scale;
}

// One warp quantises head j of one K (or V) row into a packed slot: a lane holds VPL consecutive
// elements, and stores VPL codes (VPL bytes, at a VPL-byte offset).
template <typename T, int VPL>
__device__ __forceinline__ void kv8_write_row(const T* __restrict__ src, uint8_t* __restrict__ slot_row, int32_t j,
                                              int32_t n_kv, int32_t d, int lane) {
  float x[VPL];
  float amax = 0.f;
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    x[i] = (float)src[lane * VPL + i];
    amax = fmaxf(amax, finite_abs(x[i]));
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
  const Kv8Divisor by = kv8_divisor(amax);
#pragma unroll
  for (int i = 0; i < VPL; ++i) x[i] = kv8_quotient<T>(x[i], by);
  uint8_t* dst = slot_row + (int64_t)j * d + lane * VPL;
  if constexpr (VPL % 4 == 0) {
#pragma unroll
    for (int i = 0; i < VPL; i += 4)
      *reinterpret_cast<uint32_t*>(dst + i) = f32x4_to_e4m3x4(x[i], x[i + 1], x[i + 2], x[i + 3]);
  } else {
#pragma unroll
    for (int i = 0; i < VPL; ++i) dst[i] = (uint8_t)f32x2_to_e4m3x2(x[i], 0.f);
  }
  if (lane == 0) *reinterpret_cast<float*>(slot_row + (int64_t)n_kv * d + 4 * j) = kv8_scale(amax);
}

// Rows at slots[i] (one scale per token and head): one warp per (row, head), K and V.
template <typename T, int VPL>
__global__ void __launch_bounds__(256) kv8_append_kernel(const T* __restrict__ k_new, const T* __restrict__ v_new,
                                                         const int32_t* __restrict__ slots, int32_t N,
                                                         uint8_t* __restrict__ kpool, uint8_t* __restrict__ vpool,
                                                         int32_t n_kv, int32_t d, int64_t row, int64_t n_hot,
                                                         int64_t n_slots, int32_t* err) {
  const int lane = threadIdx.x & 31;
  const int64_t total = (int64_t)N * n_kv;
  for (int64_t w = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5); w < total; w += (int64_t)gridDim.x * 8) {
    const int32_t t = (int32_t)(w / n_kv), j = (int32_t)(w % n_kv);
    const int32_t slot = slots[t];
    if (slot < n_hot || slot >= n_slots) {
      if (lane == 0) latch(err, kDevBadSlot);
      continue;
    }
    kv8_write_row<T, VPL>(k_new + w * d, kpool + (int64_t)slot * row, j, n_kv, d, lane);
    kv8_write_row<T, VPL>(v_new + w * d, vpool + (int64_t)slot * row, j, n_kv, d, lane);
  }
}

// Row b of k_new/v_new at the slot of request b's newest token (the fused append's write).
template <typename T, int VPL>
__global__ void __launch_bounds__(256) kv8_append_newest_kernel(AttnParams p) {
  const int lane = threadIdx.x & 31;
  const int64_t w = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  if (w >= (int64_t)p.B * p.n_kv) return;
  const int32_t b = (int32_t)(w / p.n_kv), j = (int32_t)(w % p.n_kv);
  int32_t n = p.reqs[b].seq_len;
  if (p.live_len) n = min(n, p.live_len[b]);
  if (n < 1) return;
  const int32_t slot = p.req_to_slot[(int64_t)b * p.cap + n - 1];
  if (slot < p.n_hot || slot >= p.n_slots) {
    if (lane == 0) latch(p.err, kDevBadSlot);
    return;
  }
  kv8_write_row<T, VPL>((const T*)p.k_new + w * p.d, (uint8_t*)p.kpool + (int64_t)slot * p.packed_row, j, p.n_kv, p.d, lane);
  kv8_write_row<T, VPL>((const T*)p.v_new + w * p.d, (uint8_t*)p.vpool + (int64_t)slot * p.packed_row, j, p.n_kv, p.d, lane);
}

template <typename T>
cudaError_t fill_t(const T* k, const T* v, int32_t L_p, uint8_t* kpool, uint8_t* vpool, int64_t first_slot,
                   int32_t n_kv, int32_t d, cudaStream_t s) {
  const int64_t ctas = (int64_t)((L_p + kPackedBlock - 1) / kPackedBlock) * n_kv;
  if (ctas > (int64_t)INT32_MAX) return cudaErrorInvalidValue;
  const dim3 grid((unsigned)ctas, 2);
  return with_vpl(d, [&](auto vpl) {
    kv8_fill_kernel<T, 32 * decltype(vpl)::value><<<grid, 256, 0, s>>>(k, v, L_p, kpool, vpool, first_slot, n_kv);
    return cudaGetLastError();
  });
}

template <typename T>
cudaError_t append_t(const T* k, const T* v, const int32_t* slots, int32_t N, uint8_t* kpool, uint8_t* vpool,
                     int32_t n_kv, int32_t d, int64_t n_hot, int64_t n_slots, int32_t* err, cudaStream_t s) {
  const int64_t ctas = ((int64_t)N * n_kv + 7) / 8;
  const unsigned grid = (unsigned)(ctas < 16384 ? ctas : 16384);
  return with_vpl(d, [&](auto vpl) {
    kv8_append_kernel<T, decltype(vpl)::value><<<grid, 256, 0, s>>>(k, v, slots, N, kpool, vpool, n_kv, d,
                                                                    kv8_row_bytes(n_kv, d), n_hot, n_slots, err);
    return cudaGetLastError();
  });
}

}  // namespace

cudaError_t launch_kv8_fill(int32_t dtype, const void* k, const void* v, int32_t L_p, uint8_t* kpool, uint8_t* vpool,
                            int64_t first_slot, int32_t n_kv, int32_t d, cudaStream_t s) {
  return dtype == 1 ? fill_t((const __nv_bfloat16*)k, (const __nv_bfloat16*)v, L_p, kpool, vpool, first_slot, n_kv, d, s)
                    : fill_t((const float*)k, (const float*)v, L_p, kpool, vpool, first_slot, n_kv, d, s);
}

cudaError_t launch_kv8_append(int32_t dtype, const void* k_new, const void* v_new, const int32_t* slots, int32_t N,
                              uint8_t* kpool, uint8_t* vpool, int32_t n_kv, int32_t d, int64_t n_hot,
                              int64_t n_slots, int32_t* err, cudaStream_t s) {
  return dtype == 1 ? append_t((const __nv_bfloat16*)k_new, (const __nv_bfloat16*)v_new, slots, N, kpool, vpool, n_kv,
                               d, n_hot, n_slots, err, s)
                    : append_t((const float*)k_new, (const float*)v_new, slots, N, kpool, vpool, n_kv, d, n_hot,
                               n_slots, err, s);
}

cudaError_t launch_kv8_append_newest(int32_t dtype, const AttnParams& p, cudaStream_t s) {
  const unsigned grid = (unsigned)(((int64_t)p.B * p.n_kv + 7) / 8);
  return with_vpl(p.d, [&](auto vpl) {
    constexpr int n = decltype(vpl)::value;
    if (dtype == 1) kv8_append_newest_kernel<__nv_bfloat16, n><<<grid, 256, 0, s>>>(p);
    else kv8_append_newest_kernel<float, n><<<grid, 256, 0, s>>>(p);
    return cudaGetLastError();
  });
}

cudaError_t launch_kv8_generic(int32_t dtype, const AttnParams& p, int32_t first_item, int32_t n_items, bool suffix,
                               cudaStream_t s, bool pdl) {
  return launch_packed_generic<8>(dtype, p, first_item, n_items, suffix, s, pdl);
}

}  // namespace granikv
