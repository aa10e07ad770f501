// hq_gemm_ep.cuh -- the single-CTA kernels with EP of hq_gemm_tile.cuh and
// their launches, shared by hq_gemm_ep.cu and hq_gemm_ep_pk.cu.
#pragma once

#include <atomic>

#include "hq_gemm_tile.cuh"

namespace hq {

// The dynamic shared-memory attribute of one kernel, set once on each device.
struct SmemAttr {
  std::atomic<unsigned long long> done{0};
  cudaError_t set(const void* fn, size_t bytes) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const unsigned long long bit = 1ull << (dev & 63);
    if (done.load(std::memory_order_relaxed) & bit) return cudaSuccess;
    e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, int(bytes));
    if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_relaxed);
    return e;
  }
};

template <int KIND, int BN, int LOGO, bool PK>
__global__ void __launch_bounds__(GemmCfg<KIND, BN, PK, true>::THREADS, 1)
    gemm_ep_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                   const __grid_constant__ CUtensorMap tmY, const __grid_constant__ CUtensorMap tmR,
                   const GemmEpParams p) {
  gemm_body<KIND, BN, LOGO, PK, true>(&tmA, &tmB, &tmY, p.residual ? &tmR : nullptr, p);
}

template <int KIND, int BN, int LOGO, bool PK>
cudaError_t launch_ep_one(const CUtensorMap* maps, const GemmEpParams& p, int grid,
                          cudaStream_t st) {
  using C = GemmCfg<KIND, BN, PK, true>;
  static SmemAttr attr;
  cudaError_t e = attr.set((const void*)gemm_ep_kernel<KIND, BN, LOGO, PK>, C::SMEM);
  if (e != cudaSuccess) return e;
  gemm_ep_kernel<KIND, BN, LOGO, PK>
      <<<grid, C::THREADS, C::SMEM, st>>>(maps[0], maps[1], maps[2], maps[3], p);
  return cudaGetLastError();
}

template <int KIND, int LOGO, bool PK>
cudaError_t launch_ep_bn(int bn, const CUtensorMap* maps, const GemmEpParams& p, int grid,
                         cudaStream_t st) {
  switch (bn) {
    case 64: return launch_ep_one<KIND, 64, LOGO, PK>(maps, p, grid, st);
    case 128: return launch_ep_one<KIND, 128, LOGO, PK>(maps, p, grid, st);
    case 192: return launch_ep_one<KIND, 192, LOGO, PK>(maps, p, grid, st);
    case 256:  // packed A's stages leave no tensor memory for 256-column tiles
      if constexpr (!PK) return launch_ep_one<KIND, 256, LOGO, PK>(maps, p, grid, st);
      return cudaErrorInvalidValue;
    default: return cudaErrorInvalidValue;
  }
}

template <bool PK>
cudaError_t launch_ep_logo(int bn, int logo, const CUtensorMap* maps, const GemmEpParams& p,
                           int grid, cudaStream_t st) {
  switch (logo) {
    case 0: return launch_ep_bn<kI8, 0, PK>(bn, maps, p, grid, st);
    case 4: return launch_ep_bn<kI8, 4, PK>(bn, maps, p, grid, st);
    case 5: return launch_ep_bn<kI8, 5, PK>(bn, maps, p, grid, st);
    case 6: return launch_ep_bn<kI8, 6, PK>(bn, maps, p, grid, st);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace hq
