// kernels_kv8_tc.cu -- tensor-core decode attention over the 8-bit cache: dense prefix items and
// COLD suffix runs, each alone or side by side in one grid (then the merge follows directly).  The
// bodies, with the design notes, are in kv8_dense_body.cuh and kv8_suffix_body.cuh.
#include "kv8_dense_body.cuh"
#include "kv8_suffix_body.cuh"

namespace granikv {
namespace {

constexpr int kSmem = k8d::kSmemBytes > k8s::kSmemBytes ? k8d::kSmemBytes : k8s::kSmemBytes;
static_assert(k8s::kThreads <= k8d::kThreads, "the suffix body runs on the dense block size");

// CTAs [0, n_dense) run dense prefix items first_dense.., CTA n_dense + k suffix token-CTA k % n_scta of
// KV-head group k / n_scta.  Dense CTA c < n_tail then runs suffix token-CTA n_scta + c (one
// KV-head group only): suffix work the plan gives the dense CTAs for after their prefix piece.
__global__ void __launch_bounds__(k8d::kThreads, 1)
    kv8_step_kernel(AttnParams p, int32_t first_dense, int32_t n_dense, const __grid_constant__ CUtensorMap tmk,
                    const __grid_constant__ CUtensorMap tmv, const int32_t* __restrict__ cta_begin, int32_t n_scta,
                    int32_t n_tail) {
  extern __shared__ __align__(128) unsigned char smem_raw[];
  const int32_t c = (int32_t)blockIdx.x;
  if (c < n_dense) {
    k8d::kv8_dense_body(p, first_dense + c, &tmk, &tmv, smem_raw);
    if (c < n_tail) {
      // the dense body has returned on every thread: its copies have landed, its MMAs have
      // completed and its tensor memory is freed, so its shared memory is free
      __syncthreads();
      fence_proxy_async_smem();
      k8s::kv8_suffix_body(p, cta_begin, n_scta + c, 0, smem_raw);
    }
  } else {
    const int32_t k = c - n_dense;
    k8s::kv8_suffix_body(p, cta_begin, k % n_scta, k / n_scta, smem_raw);
  }
}

__global__ void __launch_bounds__(k8s::kThreads, 1)
    kv8_suffix_kernel(AttnParams p, const int32_t* __restrict__ cta_begin) {
  extern __shared__ __align__(128) unsigned char smem_raw[];
  k8s::kv8_suffix_body(p, cta_begin, blockIdx.x, blockIdx.y, smem_raw);
}

}  // namespace

cudaError_t launch_kv8_step(const AttnParams& p, int32_t first_dense, int32_t n_dense, const CUtensorMap& tmk,
                            const CUtensorMap& tmv, const int32_t* cta_begin, int32_t n_scta, int32_t n_tail,
                            cudaStream_t s, bool pdl) {
  const int32_t groups = (p.n_kv + k8s::kWarps - 1) / k8s::kWarps;
  const int64_t n = (int64_t)n_dense + (int64_t)n_scta * groups;
  if (n <= 0) return cudaSuccess;
  static std::atomic<uint64_t> allowed{0};
  cudaError_t e = allow_smem_once(kv8_step_kernel, kSmem, allowed);
  if (e != cudaSuccess) return e;
  return launch_kernel(kv8_step_kernel, dim3((unsigned)n), dim3(k8d::kThreads), kSmem, s, pdl, p, first_dense, n_dense,
                       tmk, tmv, cta_begin, n_scta, n_tail);
}

cudaError_t launch_kv8_suffix(const AttnParams& p, const int32_t* cta_begin, int32_t n_scta, cudaStream_t s, bool pdl) {
  if (n_scta <= 0) return cudaSuccess;
  static std::atomic<uint64_t> allowed{0};
  cudaError_t e = allow_smem_once(kv8_suffix_kernel, k8s::kSmemBytes, allowed);
  if (e != cudaSuccess) return e;
  const dim3 grid(n_scta, (p.n_kv + k8s::kWarps - 1) / k8s::kWarps);
  return launch_kernel(kv8_suffix_kernel, grid, dim3(k8s::kThreads), k8s::kSmemBytes, s, pdl, p, cta_begin);
}

}  // namespace granikv
