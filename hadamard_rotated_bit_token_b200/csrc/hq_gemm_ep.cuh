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
                   const int has_res, const GemmEpParams p) {
  gemm_body<KIND, BN, LOGO, PK, true>(&tmA, &tmB, &tmY, has_res ? &tmR : nullptr, p);
}

template <int KIND, int BN, int LOGO, bool PK>
cudaError_t launch_ep_one(const void* tmap_a, const void* tmap_b, const void* tmap_y,
                          const void* tmap_r, const GemmEpParams& p, int grid, cudaStream_t st) {
  using C = GemmCfg<KIND, BN, PK, true>;
  static SmemAttr attr;
  cudaError_t e = attr.set((const void*)gemm_ep_kernel<KIND, BN, LOGO, PK>, C::SMEM);
  if (e != cudaSuccess) return e;
  gemm_ep_kernel<KIND, BN, LOGO, PK><<<grid, C::THREADS, C::SMEM, st>>>(
      *reinterpret_cast<const CUtensorMap*>(tmap_a), *reinterpret_cast<const CUtensorMap*>(tmap_b),
      *reinterpret_cast<const CUtensorMap*>(tmap_y),
      *reinterpret_cast<const CUtensorMap*>(tmap_r ? tmap_r : tmap_y), tmap_r ? 1 : 0, p);
  return cudaGetLastError();
}

template <int KIND, int LOGO, bool PK>
cudaError_t launch_ep_bn(int bn, const void* tmap_a, const void* tmap_b, const void* tmap_y,
                         const void* tmap_r, const GemmEpParams& p, int grid, cudaStream_t st) {
  switch (bn) {
    case 128:
      return launch_ep_one<KIND, 128, LOGO, PK>(tmap_a, tmap_b, tmap_y, tmap_r, p, grid, st);
    case 256:  // packed A's stages leave no tensor memory for 256-column tiles
      if constexpr (!PK)
        return launch_ep_one<KIND, 256, LOGO, PK>(tmap_a, tmap_b, tmap_y, tmap_r, p, grid, st);
      return cudaErrorInvalidValue;
    default:
      if constexpr (LOGO <= 5) {
        if (bn == 64)
          return launch_ep_one<KIND, 64, LOGO, PK>(tmap_a, tmap_b, tmap_y, tmap_r, p, grid, st);
        if (bn == 192)
          return launch_ep_one<KIND, 192, LOGO, PK>(tmap_a, tmap_b, tmap_y, tmap_r, p, grid, st);
      }
      return cudaErrorInvalidValue;
  }
}

template <bool PK>
cudaError_t launch_ep_logo(int bn, int logo, const void* tmap_a, const void* tmap_b,
                           const void* tmap_y, const void* tmap_r, const GemmEpParams& p, int grid,
                           cudaStream_t st) {
  switch (logo) {
    case 0: return launch_ep_bn<kI8, 0, PK>(bn, tmap_a, tmap_b, tmap_y, tmap_r, p, grid, st);
    case 4: return launch_ep_bn<kI8, 4, PK>(bn, tmap_a, tmap_b, tmap_y, tmap_r, p, grid, st);
    case 5: return launch_ep_bn<kI8, 5, PK>(bn, tmap_a, tmap_b, tmap_y, tmap_r, p, grid, st);
    case 6: return launch_ep_bn<kI8, 6, PK>(bn, tmap_a, tmap_b, tmap_y, tmap_r, p, grid, st);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace hq
