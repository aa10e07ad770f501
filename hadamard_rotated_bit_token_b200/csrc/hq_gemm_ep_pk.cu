// hq_gemm_ep_pk.cu -- the packed-code kernels of hq_gemm_ep.cu, in a
// translation unit of their own (build time).
#include "hq_gemm_ep.cuh"

namespace hq {

cudaError_t launch_gemm_ep_packed(int bn, int logo, const void* tmap_a, const void* tmap_b,
                                  const void* tmap_y, const void* tmap_r, const GemmEpParams& p,
                                  int grid, cudaStream_t st) {
  return launch_ep_logo<true>(bn, logo, tmap_a, tmap_b, tmap_y, tmap_r, p, grid, st);
}

}  // namespace hq
