// hq_gemm_ep.cu -- the products with an activation, a gate and a residual in
// their epilogue: the kernels of hq_gemm_tile.cuh with EP, for int8 codes (one
// per byte) and for bf16 operands.
#include "hq_gemm_ep.cuh"

namespace hq {

template <int KIND>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kGemmThreads, 1)
    gemm_pair_ep_kernel(const __grid_constant__ CUtensorMap tmA,
                        const __grid_constant__ CUtensorMap tmB,
                        const __grid_constant__ CUtensorMap tmY, const GemmEpParams p) {
  gemm_pair_body<KIND, true>(&tmA, &tmB, &tmY, p);
}

template <int KIND>
static cudaError_t launch_pair_kind(const CUtensorMap* maps, const GemmEpParams& p, int clusters,
                                    cudaStream_t st) {
  using C = PairCfg<KIND, true>;
  static SmemAttr attr;
  cudaError_t e = attr.set((const void*)gemm_pair_ep_kernel<KIND>, C::SMEM);
  if (e != cudaSuccess) return e;
  gemm_pair_ep_kernel<KIND>
      <<<2 * clusters, kGemmThreads, C::SMEM, st>>>(maps[0], maps[1], maps[2], p);
  return cudaGetLastError();
}

cudaError_t launch_gemm_pair_ep(bool bf16, const void* maps, const GemmEpParams& p, int clusters,
                                cudaStream_t st) {
  const CUtensorMap* m = static_cast<const CUtensorMap*>(maps);
  return bf16 ? launch_pair_kind<kBF16>(m, p, clusters, st)
              : launch_pair_kind<kI8>(m, p, clusters, st);
}

cudaError_t launch_gemm_ep(bool bf16, int bn, int logo, bool packed_a, const void* maps,
                           const GemmEpParams& p, int grid, cudaStream_t st) {
  if (packed_a) return launch_gemm_ep_packed(bn, logo, maps, p, grid, st);
  const CUtensorMap* m = static_cast<const CUtensorMap*>(maps);
  if (bf16) return launch_ep_bn<kBF16, 0, false>(bn, m, p, grid, st);
  return launch_ep_logo<false>(bn, logo, m, p, grid, st);
}

}  // namespace hq
