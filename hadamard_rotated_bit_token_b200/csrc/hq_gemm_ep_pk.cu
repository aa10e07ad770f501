// hq_gemm_ep_pk.cu -- the packed-code kernels of hq_gemm_ep.cu, in a
// translation unit of their own (build time).
#include "hq_gemm_ep.cuh"

namespace hq {

cudaError_t launch_gemm_ep_packed(int bn, int logo, const void* maps, const GemmEpParams& p,
                                  int grid, cudaStream_t st) {
  return launch_ep_logo<true>(bn, logo, static_cast<const CUtensorMap*>(maps), p, grid, st);
}

}  // namespace hq
