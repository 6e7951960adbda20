// kernels_kv4.cu -- 4-bit cache: the kernels that quantise K/V rows into packed slots, and the launch of the
// CUDA-core decode attention over such slots (packed_generic_body.cuh).
#include "kv4_util.cuh"
#include "launch_util.cuh"
#include "packed_generic_body.cuh"

namespace granikv {
namespace {

// One block of kPackedBlock slab tokens of one KV head, of K (blockIdx.y = 0) or V.  A thread holds groups of 16
// elements in registers between the block's amax and their codes, so the rows are read once: 2.6 bytes moved for
// each bf16 element.  Bound by memory: 16K tokens of 8 x 128 take 18.4 us from bf16 (86 MB, 0.69 of the copy rate) and
// 25.6 from fp32 (0.88); without the quantising, the same loads and stores of bf16 take 17.3.  (With two
// loads of 16 bytes in place of one of 32 and a quotient an instruction instead of two: 21.0 us.)
template <typename T, int D, bool WIDE>
__global__ void __launch_bounds__(256) kv4_fill_kernel(const T* __restrict__ k, const T* __restrict__ v, int32_t L_p,
                                                       uint8_t* __restrict__ kpool, uint8_t* __restrict__ vpool,
                                                       int64_t first_slot, int32_t n_kv) {
  constexpr int kPerRow = D / kKv4Group;                    // groups of a head's row
  constexpr int kGroups = kPackedBlock * kPerRow;              // of the block
  constexpr int kPer = (kGroups + 255) / 256;               // of a thread
  __shared__ float s_max[8];
  const int32_t j = blockIdx.x % n_kv;
  const int32_t t0 = blockIdx.x / n_kv * kPackedBlock;
  const int32_t n = min(kPackedBlock, L_p - t0);
  const T* src = (blockIdx.y ? v : k) + ((int64_t)t0 * n_kv + j) * D;
  Kv4Group<T> x[kPer];
#pragma unroll
  for (int c = 0; c < kPer; ++c) {
    const int32_t idx = threadIdx.x + c * 256, t = idx / kPerRow;
    if (idx < kGroups && t < n) x[c].template load<WIDE>(src + (int64_t)t * (n_kv * D) + idx % kPerRow * kKv4Group);
    else x[c].clear();
  }
  float top[kPer], finite[kPer], amax = 0.f;
#pragma unroll
  for (int c = 0; c < kPer; ++c) {
    top[c] = x[c].top();
    finite[c] = kv4_finite_top(x[c], top[c]);
    amax = fmaxf(amax, finite[c]);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
  if ((threadIdx.x & 31) == 0) s_max[threadIdx.x >> 5] = amax;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < 8; ++w) amax = fmaxf(amax, s_max[w]);
  const uint32_t byte = kv4_exponent(amax);
  const int64_t row = kv4_row_bytes(n_kv, D);
  uint8_t* dst = (blockIdx.y ? vpool : kpool) + (first_slot + t0) * row;
  const int64_t codes = (int64_t)j * (D / 2), scales = kv4_scales_at(n_kv, D) + (int64_t)j * kPerRow, unit = kv4_units_at(n_kv, D) + j;
#pragma unroll
  for (int c = 0; c < kPer; ++c) {
    const int32_t idx = threadIdx.x + c * 256, t = idx / kPerRow;
    if (idx < kGroups && t < n) {
      uint32_t scale;
      const uint2 w = kv4_codes(x[c], top[c], finite[c], byte, scale);
      uint8_t* at = dst + t * row;
      *reinterpret_cast<uint2*>(at + codes + idx % kPerRow * 8) = w;
      at[scales + idx % kPerRow] = (uint8_t)scale;
    }
  }
  for (int32_t t = threadIdx.x; t < n; t += 256) dst[t * row + unit] = (uint8_t)byte;
}

// Single tokens: a team of lanes, a group of 16 elements each, takes one head of a token's K or V.
template <int D>
constexpr int kv4_team() {
  return D / kKv4Group <= 2 ? 2 : D / kKv4Group <= 4 ? 4 : D / kKv4Group <= 8 ? 8 : 16;
}

// src: the head's elements, slot_row: its packed row, or NULL (the team then only takes part in the exchange)
template <typename T, int D>
__device__ __forceinline__ void kv4_write_row(const T* __restrict__ src, uint8_t* __restrict__ slot_row, int32_t j, int32_t n_kv) {
  constexpr int kTeam = kv4_team<D>();
  const int i = threadIdx.x % kTeam;
  const bool mine = slot_row && i < D / kKv4Group;
  Kv4Group<T> x;
  if (mine) x.template load<false>(src + i * kKv4Group);
  else x.clear();
  const float top = x.top(), finite = kv4_finite_top(x, top);
  float amax = finite;
#pragma unroll
  for (int o = kTeam / 2; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
  const uint32_t byte = kv4_exponent(amax);
  uint32_t scale;
  const uint2 w = kv4_codes(x, top, finite, byte, scale);
  if (!mine) return;
  *reinterpret_cast<uint2*>(slot_row + (int64_t)j * (D / 2) + i * 8) = w;
  slot_row[kv4_scales_at(n_kv, D) + (int64_t)j * (D / kKv4Group) + i] = (uint8_t)scale;
  if (i == 0) slot_row[kv4_units_at(n_kv, D) + j] = (uint8_t)byte;
}

// Rows at slots[i]: 16K tokens of 8 x 128 from bf16 20.9 us, from fp32 25.5.  Item w is head w / 2 % n_kv of token w / 2 / n_kv, its K (w even) or V.
template <typename T, int D>
__global__ void __launch_bounds__(256) kv4_append_kernel(const T* __restrict__ k_new, const T* __restrict__ v_new,
                                                         const int32_t* __restrict__ slots, int32_t N,
                                                         uint8_t* __restrict__ kpool, uint8_t* __restrict__ vpool,
                                                         int32_t n_kv, int64_t n_hot, int64_t n_slots, int32_t* err) {
  constexpr int kTeam = kv4_team<D>(), kItems = 256 / kTeam;
  const int64_t total = (int64_t)N * n_kv * 2, row = kv4_row_bytes(n_kv, D);
  // (whole warps stay in the loop: the team's exchange names every lane)
  for (int64_t w0 = (int64_t)blockIdx.x * kItems; w0 < total; w0 += (int64_t)gridDim.x * kItems) {
    const int64_t w = w0 + threadIdx.x / kTeam;
    uint8_t* at = nullptr;
    const T* src = nullptr;
    int32_t j = 0;
    if (w < total) {
      const int64_t h = w / 2;
      const int32_t t = (int32_t)(h / n_kv), slot = slots[t];
      j = (int32_t)(h - (int64_t)t * n_kv);
      src = (w & 1 ? v_new : k_new) + h * D;
      if (slot >= n_hot && slot < n_slots) at = (w & 1 ? vpool : kpool) + slot * row;
      else latch(err, kDevBadSlot);
    }
    kv4_write_row<T, D>(src, at, j, n_kv);
  }
}

// Row b of k_new/v_new at the slot of request b's newest token (the fused append's write).  Launched as a dependent of
// what the stream ran before, and the attention as a dependent of this: its set-up overlaps the writes, and it reads
// nothing that they change before this grid is done.
template <typename T, int D>
__global__ void __launch_bounds__(256) kv4_append_newest_kernel(AttnParams p) {
  constexpr int kTeam = kv4_team<D>(), kItems = 256 / kTeam;
  const int64_t w = (int64_t)blockIdx.x * kItems + threadIdx.x / kTeam;
  uint8_t* at = nullptr;
  const T* src = nullptr;
  int32_t j = 0;
  grid_dep_launch_dependents();
  grid_dep_wait();
  if (w < (int64_t)p.B * p.n_kv * 2) {
    const int64_t h = w / 2;
    const int32_t b = (int32_t)(h / p.n_kv);
    j = (int32_t)(h - (int64_t)b * p.n_kv);
    src = (const T*)(w & 1 ? p.v_new : p.k_new) + h * D;
    int32_t n = p.reqs[b].seq_len;
    if (p.live_len) n = min(n, p.live_len[b]);
    if (n >= 1) {
      const int32_t slot = p.req_to_slot[(int64_t)b * p.cap + n - 1];
      if (slot >= p.n_hot && slot < p.n_slots) at = (uint8_t*)(w & 1 ? p.vpool : p.kpool) + slot * p.packed_row;
      else latch(p.err, kDevBadSlot);
    }
  }
  kv4_write_row<T, D>(src, at, j, p.n_kv);
}

template <typename T>
cudaError_t fill_t(const T* k, const T* v, int32_t L_p, uint8_t* kpool, uint8_t* vpool, int64_t first_slot,
                   int32_t n_kv, int32_t d, cudaStream_t s) {
  const int64_t ctas = (int64_t)((L_p + kPackedBlock - 1) / kPackedBlock) * n_kv;
  if (ctas > (int64_t)INT32_MAX) return cudaErrorInvalidValue;
  const dim3 grid((unsigned)ctas, 2);
  return with_vpl(d, [&](auto vpl) {
    constexpr int D = 32 * decltype(vpl)::value;
    auto kernel = ((uintptr_t)k | (uintptr_t)v) % 32 ? kv4_fill_kernel<T, D, false> : kv4_fill_kernel<T, D, true>;
    kernel<<<grid, 256, 0, s>>>(k, v, L_p, kpool, vpool, first_slot, n_kv);
    return cudaGetLastError();
  });
}

template <typename T>
cudaError_t append_t(const T* k, const T* v, const int32_t* slots, int32_t N, uint8_t* kpool, uint8_t* vpool,
                     int32_t n_kv, int32_t d, int64_t n_hot, int64_t n_slots, int32_t* err, cudaStream_t s) {
  return with_vpl(d, [&](auto vpl) {
    constexpr int D = 32 * decltype(vpl)::value, kItems = 256 / kv4_team<D>();
    const int64_t ctas = ((int64_t)N * n_kv * 2 + kItems - 1) / kItems;
    const unsigned grid = (unsigned)(ctas < 65536 ? ctas : 65536);
    kv4_append_kernel<T, D><<<grid, 256, 0, s>>>(k, v, slots, N, kpool, vpool, n_kv, n_hot, n_slots, err);
    return cudaGetLastError();
  });
}

}  // namespace

cudaError_t launch_kv4_fill(int32_t dtype, const void* k, const void* v, int32_t L_p, uint8_t* kpool, uint8_t* vpool,
                            int64_t first_slot, int32_t n_kv, int32_t d, cudaStream_t s) {
  return dtype == 1 ? fill_t((const __nv_bfloat16*)k, (const __nv_bfloat16*)v, L_p, kpool, vpool, first_slot, n_kv, d, s)
                    : fill_t((const float*)k, (const float*)v, L_p, kpool, vpool, first_slot, n_kv, d, s);
}

cudaError_t launch_kv4_append(int32_t dtype, const void* k_new, const void* v_new, const int32_t* slots, int32_t N,
                              uint8_t* kpool, uint8_t* vpool, int32_t n_kv, int32_t d, int64_t n_hot,
                              int64_t n_slots, int32_t* err, cudaStream_t s) {
  return dtype == 1 ? append_t((const __nv_bfloat16*)k_new, (const __nv_bfloat16*)v_new, slots, N, kpool, vpool, n_kv,
                               d, n_hot, n_slots, err, s)
                    : append_t((const float*)k_new, (const float*)v_new, slots, N, kpool, vpool, n_kv, d, n_hot,
                               n_slots, err, s);
}

cudaError_t launch_kv4_append_newest(int32_t dtype, const AttnParams& p, cudaStream_t s) {
  return with_vpl(p.d, [&](auto vpl) {
    constexpr int D = 32 * decltype(vpl)::value, kItems = 256 / kv4_team<D>();
    const unsigned grid = (unsigned)(((int64_t)p.B * p.n_kv * 2 + kItems - 1) / kItems);
    auto kernel = dtype == 1 ? kv4_append_newest_kernel<__nv_bfloat16, D> : kv4_append_newest_kernel<float, D>;
    return launch_kernel(kernel, dim3(grid), dim3(256), 0, s, true, p);
  });
}

cudaError_t launch_kv4_generic(int32_t dtype, const AttnParams& p, int32_t first_item, int32_t n_items, bool suffix,
                               cudaStream_t s, bool pdl) {
  return launch_packed_generic<4>(dtype, p, first_item, n_items, suffix, s, pdl);
}

}  // namespace granikv
