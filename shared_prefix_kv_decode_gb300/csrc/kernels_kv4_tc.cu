// kernels_kv4_tc.cu -- the tensor-core decode step of packed_step_body.cuh over the 4-bit cache.
#include "packed_step_body.cuh"

namespace granikv {

cudaError_t launch_kv4_step(const AttnParams& p, int32_t first_dense, int32_t n_dense, const PackedMaps& m,
                            const int32_t* cta_begin, int32_t n_scta, int32_t n_tail, cudaStream_t s, bool pdl) {
  const auto launch = p.d == 64 ? launch_packed_step<4, 64> : launch_packed_step<4, 128>;
  return launch(p, first_dense, n_dense, m, cta_begin, n_scta, n_tail, s, pdl);
}

cudaError_t launch_kv4_suffix(const AttnParams& p, const int32_t* cta_begin, int32_t n_scta, cudaStream_t s, bool pdl) {
  return (p.d == 64 ? launch_packed_suffix<4, 64> : launch_packed_suffix<4, 128>)(p, cta_begin, n_scta, s, pdl);
}

}  // namespace granikv
