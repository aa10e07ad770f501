// hq_gemm_ep.cu -- the products with an activation, a gate and a residual in
// their epilogue: the kernels of hq_gemm_tile.cuh with EP, for int8 codes (one
// per byte) and for bf16 operands.
#include "hq_gemm_ep.cuh"

namespace hq {

template <int KIND>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kGemmThreads, 1)
    gemm_pair_ep_kernel(const __grid_constant__ CUtensorMap tmA,
                        const __grid_constant__ CUtensorMap tmB,
                        const __grid_constant__ CUtensorMap tmY,
                        const __grid_constant__ CUtensorMap tmR, const int has_res,
                        const GemmEpParams p) {
  gemm_pair_body<KIND, true>(&tmA, &tmB, &tmY, has_res ? &tmR : nullptr, p);
}

template <int KIND>
static cudaError_t launch_pair_kind(const void* tmap_a, const void* tmap_b, const void* tmap_y,
                                    const void* tmap_r, const GemmEpParams& p, int clusters,
                                    cudaStream_t st) {
  using C = PairCfg<KIND, true>;
  static SmemAttr attr;
  cudaError_t e = attr.set((const void*)gemm_pair_ep_kernel<KIND>, C::SMEM);
  if (e != cudaSuccess) return e;
  gemm_pair_ep_kernel<KIND><<<2 * clusters, kGemmThreads, C::SMEM, st>>>(
      *reinterpret_cast<const CUtensorMap*>(tmap_a), *reinterpret_cast<const CUtensorMap*>(tmap_b),
      *reinterpret_cast<const CUtensorMap*>(tmap_y),
      *reinterpret_cast<const CUtensorMap*>(tmap_r ? tmap_r : tmap_y), tmap_r ? 1 : 0, p);
  return cudaGetLastError();
}

cudaError_t launch_gemm_pair_ep(bool bf16, const void* tmap_a, const void* tmap_b,
                                const void* tmap_y, const void* tmap_r, const GemmEpParams& p,
                                int clusters, cudaStream_t st) {
  return bf16 ? launch_pair_kind<kBF16>(tmap_a, tmap_b, tmap_y, tmap_r, p, clusters, st)
              : launch_pair_kind<kI8>(tmap_a, tmap_b, tmap_y, tmap_r, p, clusters, st);
}

cudaError_t launch_gemm_ep(bool bf16, int bn, int logo, bool packed_a, const void* tmap_a,
                           const void* tmap_b, const void* tmap_y, const void* tmap_r,
                           const GemmEpParams& p, int grid, cudaStream_t st) {
  if (packed_a) return launch_gemm_ep_packed(bn, logo, tmap_a, tmap_b, tmap_y, tmap_r, p, grid, st);
  if (bf16) return launch_ep_bn<kBF16, 0, false>(bn, tmap_a, tmap_b, tmap_y, tmap_r, p, grid, st);
  return launch_ep_logo<false>(bn, logo, tmap_a, tmap_b, tmap_y, tmap_r, p, grid, st);
}

}  // namespace hq
