// hq_gemm_ep.cu -- the products with an activation, a gate and a residual in
// their epilogue: the kernels of hq_gemm_tile.cuh with EP, for int8 codes (one
// per byte) and for bf16 operands.
#include "hq_gemm_ep.cuh"

namespace hq {

template <int KIND, int BN>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(PairCfg<KIND, BN, true>::THREADS, 1)
    gemm_pair_ep_kernel(const __grid_constant__ CUtensorMap tmA,
                        const __grid_constant__ CUtensorMap tmB,
                        const __grid_constant__ CUtensorMap tmY,
                        const __grid_constant__ CUtensorMap tmR, const GemmEpParams p) {
  gemm_pair_body<KIND, BN, true>(&tmA, &tmB, &tmY, p.residual ? &tmR : nullptr, p);
}

template <int KIND, int BN>
static cudaError_t launch_pair_one(const CUtensorMap* maps, const GemmEpParams& p, int clusters,
                                   cudaStream_t st) {
  using C = PairCfg<KIND, BN, true>;
  static SmemAttr attr;
  cudaError_t e = attr.set((const void*)gemm_pair_ep_kernel<KIND, BN>, C::SMEM);
  if (e != cudaSuccess) return e;
  gemm_pair_ep_kernel<KIND, BN>
      <<<2 * clusters, C::THREADS, C::SMEM, st>>>(maps[0], maps[1], maps[2], maps[3], p);
  return cudaGetLastError();
}

template <int KIND>
static cudaError_t launch_pair_kind(int bn, const CUtensorMap* maps, const GemmEpParams& p,
                                    int clusters, cudaStream_t st) {
  switch (bn) {
    case 128: return launch_pair_one<KIND, 128>(maps, p, clusters, st);
    case 192: return launch_pair_one<KIND, 192>(maps, p, clusters, st);
    default: return launch_pair_one<KIND, 256>(maps, p, clusters, st);
  }
}

cudaError_t launch_gemm_pair_ep(bool bf16, int bn, const void* maps, const GemmEpParams& p,
                                int clusters, cudaStream_t st) {
  const CUtensorMap* m = static_cast<const CUtensorMap*>(maps);
  return bf16 ? launch_pair_kind<kBF16>(bn, m, p, clusters, st)
              : launch_pair_kind<kI8>(bn, m, p, clusters, st);
}

cudaError_t launch_gemm_ep(bool bf16, int bn, int logo, bool packed_a, const void* maps,
                           const GemmEpParams& p, int grid, cudaStream_t st) {
  if (packed_a) return launch_gemm_ep_packed(bn, logo, maps, p, grid, st);
  const CUtensorMap* m = static_cast<const CUtensorMap*>(maps);
  if (bf16) return launch_ep_bn<kBF16, 0, false>(bn, m, p, grid, st);
  return launch_ep_logo<false>(bn, logo, m, p, grid, st);
}

}  // namespace hq
