// packed_step_body.cuh -- tensor-core decode attention over an 8- or 4-bit cache: dense prefix items and
// COLD suffix runs, each alone or side by side in one grid (then the merge follows directly).  The
// bodies, with the design notes, are in packed_dense_body.cuh and packed_suffix_body.cuh.
#pragma once

#include "packed_dense_body.cuh"
#include "packed_suffix_body.cuh"

namespace granikv {
namespace {

template <int BITS, int D>
constexpr int kStepSmem = pkd::Layout<BITS, D>::kSmemBytes > pks::Layout<BITS, D>::kSmemBytes ? pkd::Layout<BITS, D>::kSmemBytes
                                                                                             : pks::Layout<BITS, D>::kSmemBytes;
static_assert(pks::kThreads <= pkd::Layout<8, 128>::kThreads && pks::kThreads <= pkd::Layout<4, 128>::kThreads, "the suffix body runs on the dense block size");

// CTAs [0, n_dense) run dense prefix items first_dense.., CTA n_dense + k suffix token-CTA k % n_scta of
// KV-head group k / n_scta.  Dense CTA c < n_tail then runs suffix token-CTA n_scta + c (one
// KV-head group only): suffix work the plan gives the dense CTAs for after their prefix piece.
template <int BITS, int D>
__global__ void __launch_bounds__(pkd::Layout<BITS, D>::kThreads, 1)
    packed_step_kernel(AttnParams p, int32_t first_dense, int32_t n_dense, const __grid_constant__ PackedMaps maps,
                       const int32_t* __restrict__ cta_begin, int32_t n_scta, int32_t n_tail) {
  extern __shared__ __align__(128) unsigned char smem_raw[];
  const int32_t c = (int32_t)blockIdx.x;
  if (c < n_dense) {
    pkd::packed_dense_body<BITS, D>(p, first_dense + c, &maps, smem_raw);
    if (c < n_tail) {
      // the dense body has returned on every thread: its copies have landed, its MMAs have
      // completed and its tensor memory is freed, so its shared memory is free
      __syncthreads();
      fence_proxy_async_smem();
      pks::packed_suffix_body<BITS, D, pkd::Layout<BITS, D>::kSplitRegs>(p, cta_begin, n_scta + c, 0, smem_raw);
    }
  } else {
    const int32_t k = c - n_dense;
    pks::packed_suffix_body<BITS, D, pkd::Layout<BITS, D>::kSplitRegs>(p, cta_begin, k % n_scta, k / n_scta, smem_raw);
  }
}

template <int BITS, int D>
__global__ void __launch_bounds__(pks::kThreads, 1) packed_suffix_kernel(AttnParams p, const int32_t* __restrict__ cta_begin) {
  extern __shared__ __align__(128) unsigned char smem_raw[];
  pks::packed_suffix_body<BITS, D, false>(p, cta_begin, blockIdx.x, blockIdx.y, smem_raw);
}

template <int BITS, int D>
cudaError_t launch_packed_step(const AttnParams& p, int32_t first_dense, int32_t n_dense, const PackedMaps& maps,
                               const int32_t* cta_begin, int32_t n_scta, int32_t n_tail, cudaStream_t s, bool pdl) {
  const int32_t groups = (p.n_kv + pks::kWarps - 1) / pks::kWarps;
  const int64_t n = (int64_t)n_dense + (int64_t)n_scta * groups;
  if (n <= 0) return cudaSuccess;
  if (n > (int64_t)INT32_MAX) return cudaErrorInvalidValue;
  static std::atomic<uint64_t> allowed{0};
  cudaError_t e = allow_smem_once(packed_step_kernel<BITS, D>, kStepSmem<BITS, D>, allowed);
  if (e != cudaSuccess) return e;
  return launch_kernel(packed_step_kernel<BITS, D>, dim3((unsigned)n), dim3(pkd::Layout<BITS, D>::kThreads), kStepSmem<BITS, D>, s, pdl, p, first_dense,
                       n_dense, maps, cta_begin, n_scta, n_tail);
}

template <int BITS, int D>
cudaError_t launch_packed_suffix(const AttnParams& p, const int32_t* cta_begin, int32_t n_scta, cudaStream_t s, bool pdl) {
  if (n_scta <= 0) return cudaSuccess;
  static std::atomic<uint64_t> allowed{0};
  constexpr int smem = pks::Layout<BITS, D>::kSmemBytes;
  cudaError_t e = allow_smem_once(packed_suffix_kernel<BITS, D>, smem, allowed);
  if (e != cudaSuccess) return e;
  const dim3 grid(n_scta, (p.n_kv + pks::kWarps - 1) / pks::kWarps);
  return launch_kernel(packed_suffix_kernel<BITS, D>, grid, dim3(pks::kThreads), smem, s, pdl, p, cta_begin);
}

}  // namespace
}  // namespace granikv
