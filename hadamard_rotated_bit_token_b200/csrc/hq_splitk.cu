// hq_splitk.cu -- the products with an epilogue when the output has too few
// tiles to fill the GPU: K split over a cluster of CTAs.
//
//   z[t,n] = sum_k A[t,k] B[n,k],  Y[t,n] = bf16(R + g * act(epilogue(z)))
//
// A cluster of p.split CTAs computes 128 weight rows x NT tokens; each CTA takes
// a run of 128-byte K blocks.  The weights are the MMA's M side (128 rows) and
// the tokens its N side, so a batch of 16 tokens costs 16 columns of tensor
// memory and of shared memory, not a tile of 128.  Warp 0 loads (TMA, 128-byte
// swizzle, a ring of stages), warp 1 issues tcgen05.mma (kind::f16 or kind::i8)
// into NT columns of tensor memory, warps 2..5 write the CTA's partial sums
// [token][weight row] into shared memory over the spent stages.  After a cluster
// barrier each CTA adds the split's partial sums, always in rank order, for its
// share of the tokens through distributed shared memory, applies the epilogue
// and stores.  Integer sums are exact; fp32 sums depend on the sizes alone.
//
// Without the split a narrow layer is a few CTAs that walk all of K: 64 tokens,
// K = 4608, N = 1152 in bf16 took 23.3 us by tiles of 128 x 192 on 6 SMs; by 9
// clusters of 8 CTAs see splitk_plan.
#include <cuda.h>
#include <cuda_bf16.h>

#include <atomic>

#include "hq_act.cuh"
#include "hq_device.cuh"
#include "hq_kernels.h"

namespace hq {

namespace {

constexpr int kSkRows = 128;     // weight rows per tile (MMA M)
constexpr int kSkThreads = 192;  // producer, MMA issuer, four epilogue warps
constexpr int kSkI8 = 0, kSkBF16 = 1;

// D format at bits 4-5 (s32 2, fp32 1), operand formats 1 (int8, bf16) at bits
// 7-9 and 10-12, N >> 3 at bits 17-22, M >> 4 at bits 24-28.
template <int KIND>
constexpr uint32_t sk_idesc(int n) {
  return (KIND == kSkBF16 ? 1u << 4 : 2u << 4) | (1u << 7) | (1u << 10) | (uint32_t(n >> 3) << 17) |
         (uint32_t(kSkRows >> 4) << 24);
}

__device__ __forceinline__ uint64_t sk_desc(uint32_t saddr) {
  // K-major, rows of 128 bytes, 128-byte swizzle (8-row atoms of 1024 bytes)
  return uint64_t((saddr & 0x3FFFFu) >> 4) | (uint64_t(1) << 16) | (uint64_t(1024 >> 4) << 32) |
         (uint64_t(1) << 46) | (uint64_t(2) << 61);
}

template <int NT>
struct SkCfg {
  static constexpr int W_BYTES = kSkRows * 128;
  static constexpr int X_BYTES = NT * 128;
  static constexpr int STAGE_BYTES = W_BYTES + X_BYTES;
  // two CTAs an SM
  static constexpr int STAGES = (110 * 1024) / STAGE_BYTES;
  static constexpr int TMEM_COLS = NT < 32 ? 32 : NT;
  static constexpr int PART_BYTES = NT * kSkRows * 4;
  static constexpr size_t SMEM = size_t(STAGES) * STAGE_BYTES + 256 + 1024;
  static_assert(PART_BYTES <= STAGES * STAGE_BYTES, "partial sums fit the stages");
  static_assert(X_BYTES % 1024 == 0, "stage bases stay 1024-byte aligned");
  static_assert(16 * STAGES + 32 <= 256, "barrier block");
};

__device__ __forceinline__ float2 ld_cluster_f2(uint32_t addr) {
  float2 v;
  asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(addr));
  return v;
}

__device__ __forceinline__ float2 bf16x2_at(const uint16_t* p) {
  return unpack_bf16x2(*reinterpret_cast<const uint32_t*>(p));
}

}  // namespace

template <int KIND, int NT>
__global__ void __launch_bounds__(kSkThreads, 2)
    splitk_kernel(const __grid_constant__ CUtensorMap tmX, const __grid_constant__ CUtensorMap tmW,
                  const SplitKParams p) {
  using C = SkCfg<NT>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint8_t* sW = smem;
  uint8_t* sX = smem + size_t(C::STAGES) * C::W_BYTES;
  float* part = reinterpret_cast<float*>(smem);  // [NT][kSkRows], over the stages
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + size_t(C::STAGES) * C::STAGE_BYTES);
  uint64_t* empty = full + C::STAGES;
  uint64_t* tfull = empty + C::STAGES;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(tfull + 1);
  volatile int* failed = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const WaitCtl wc{p.err, p.wait_ns};
  const int rank = int(cluster_ctarank());
  const int tile = int(blockIdx.x) / p.split;
  const int n0 = (tile % p.num_n_tiles) * kSkRows;
  const int t0 = (tile / p.num_n_tiles) * NT;
  const int kb0 = int(int64_t(p.k_blocks) * rank / p.split);
  const int kb1 = int(int64_t(p.k_blocks) * (rank + 1) / p.split);

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::STAGES; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    mbar_init(tfull, 1);
    *failed = 0;
    fence_mbarrier_init();
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, C::TMEM_COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  if (warp == 0) {
    if (lane == 0) {
      int stage = 0, issued = 0;
      uint32_t phase = 0;
      for (int kb = kb0; kb < kb1; ++kb) {
        if (*failed || !mbar_wait(&empty[stage], phase ^ 1u, wc)) {
          *failed = 1;
          break;
        }
        mbar_arrive_expect_tx(&full[stage], C::STAGE_BYTES);
        tma_load_2d(sW + size_t(stage) * C::W_BYTES, &tmW, kb * 128, n0, &full[stage]);
        tma_load_2d(sX + size_t(stage) * C::X_BYTES, &tmX, kb * 128, t0, &full[stage]);
        ++issued;
        if (++stage == C::STAGES) {
          stage = 0;
          phase ^= 1u;
        }
      }
      if (*failed) {
        // the copies in flight land before the CTA can exit
        for (int i = 0; i < C::STAGES && i < issued; ++i) {
          if (--stage < 0) {
            stage = C::STAGES - 1;
            phase ^= 1u;
          }
          (void)mbar_wait(&full[stage], phase, wc);
        }
      }
    }
  } else if (warp == 1) {
    if (lane == 0) {
      int stage = 0;
      uint32_t phase = 0;
      const uint32_t w_base = smem_u32(sW), x_base = smem_u32(sX);
      for (int kb = kb0; kb < kb1; ++kb) {
        if (*failed || !mbar_wait(&full[stage], phase, wc)) {
          *failed = 1;
          break;
        }
        tc_fence_after();
        const uint64_t wd = sk_desc(w_base + uint32_t(stage) * C::W_BYTES);
        const uint64_t xd = sk_desc(x_base + uint32_t(stage) * C::X_BYTES);
#pragma unroll
        for (int k = 0; k < 4; ++k) {  // 32 bytes along K inside the swizzle row
          if constexpr (KIND == kSkBF16)
            mma_bf16(tmem, wd + uint64_t(2 * k), xd + uint64_t(2 * k), sk_idesc<KIND>(NT),
                     (kb > kb0 || k > 0) ? 1u : 0u);
          else
            mma_i8(tmem, wd + uint64_t(2 * k), xd + uint64_t(2 * k), sk_idesc<KIND>(NT),
                   (kb > kb0 || k > 0) ? 1u : 0u);
        }
        mma_commit(&empty[stage]);
        if (++stage == C::STAGES) {
          stage = 0;
          phase ^= 1u;
        }
      }
      mma_commit(tfull);  // every MMA issued has completed
      (void)mbar_wait(tfull, 0, wc);
    }
  } else {
    // lane quarter warp % 4 of tensor memory: weight rows 32 q + lane
    const bool got = mbar_wait(tfull, 0, wc);
    if (__all_sync(0xffffffffu, got) && !*failed) {
      tc_fence_after();
      const int q = warp & 3;
      float* dst = part + q * 32 + lane;
#pragma unroll
      for (int c = 0; c < NT; c += 32) {
        uint32_t r[32];
        tmem_ld_32x32b_x32(tmem + (uint32_t(q * 32) << 16) + uint32_t(c), r);
        tmem_wait_ld();
#pragma unroll
        for (int i = 0; i < 32; ++i)
          if (c + i < NT) dst[(c + i) * kSkRows] = __uint_as_float(r[i]);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // every CTA's partial sums are in place

  if (!*failed) {
    // pairs of weight rows of this CTA's share of the tokens
    const int tb = NT * rank / p.split, te = NT * (rank + 1) / p.split;
    for (int i = int(threadIdx.x); i < (te - tb) * (kSkRows / 2); i += kSkThreads) {
      const int tt = tb + i / (kSkRows / 2), j = 2 * (i % (kSkRows / 2));
      const int t = t0 + tt, n = n0 + j;
      if (t >= p.T || n >= p.N) continue;
      const float* src = part + tt * kSkRows + j;
      f2 z;
      if constexpr (KIND == kSkBF16) {
        f2 v = ld_cluster_f2(mapa_shared(src, 0));
#pragma unroll 4
        for (int k = 1; k < p.split; ++k) v = add2(v, ld_cluster_f2(mapa_shared(src, uint32_t(k))));
        z = p.bias16 ? add2(v, bf16x2_at(p.bias16 + n)) : v;
      } else {
        int a = 0, b = 0;
#pragma unroll 4
        for (int k = 0; k < p.split; ++k) {
          const f2 v = ld_cluster_f2(mapa_shared(src, uint32_t(k)));
          a += __float_as_int(v.x);
          b += __float_as_int(v.y);
        }
        const float sx = p.a_scale_per_row ? p.a_scale[t] : p.a_scale[0];
        const float2 sw = *reinterpret_cast<const float2*>(p.w_scale + n);
        f2 c = p.bias ? *reinterpret_cast<const float2*>(p.bias + n) : pk(0.0f, 0.0f);
        if (p.a_mean) {
          const float m = p.a_mean[t];
          c = fma2(pk(m, m), *reinterpret_cast<const float2*>(p.colsum + n), c);
        }
        z = fma2(pk(__int2float_rn(a), __int2float_rn(b)), mul2(pk(sx, sx), sw), c);
      }
      f2 zz[1] = {z};
      act_chunk(p.act, zz);
      z = zz[0];
      const int64_t off = int64_t(t) * p.N + n;
      if (p.gate) z = mul2(z, bf16x2_at(p.gate + (t / p.gate_rows) * p.N + n));
      if (p.residual) z = add2(z, bf16x2_at(p.residual + off));
      *reinterpret_cast<uint32_t*>(p.Y + off) = pack_bf16x2(z.x, z.y);
    }
  }
  cluster_sync();  // no CTA leaves while a peer may read its partial sums
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, C::TMEM_COLS);
  }
}

namespace {

template <int KIND, int NT>
cudaError_t launch_one(const void* tmap_x, const void* tmap_w, const SplitKParams& p, int tiles,
                       cudaStream_t st) {
  using C = SkCfg<NT>;
  const void* fn = (const void*)splitk_kernel<KIND, NT>;
  static std::atomic<unsigned long long> done{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const unsigned long long bit = 1ull << (dev & 63);
  if (!(done.load(std::memory_order_relaxed) & bit)) {
    e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, int(C::SMEM));
    if (e == cudaSuccess)
      e = cudaFuncSetAttribute(fn, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
    done.fetch_or(bit, std::memory_order_relaxed);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(tiles) * unsigned(p.split));
  cfg.blockDim = dim3(kSkThreads);
  cfg.dynamicSmemBytes = C::SMEM;
  cfg.stream = st;
  cudaLaunchAttribute a[1];
  a[0].id = cudaLaunchAttributeClusterDimension;
  a[0].val.clusterDim.x = unsigned(p.split);
  a[0].val.clusterDim.y = 1;
  a[0].val.clusterDim.z = 1;
  cfg.attrs = a;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, splitk_kernel<KIND, NT>,
                            *static_cast<const CUtensorMap*>(tmap_x),
                            *static_cast<const CUtensorMap*>(tmap_w), p);
}

template <int KIND>
cudaError_t launch_nt(int nt, const void* tmap_x, const void* tmap_w, const SplitKParams& p,
                      int tiles, cudaStream_t st) {
  switch (nt) {
    case 16: return launch_one<KIND, 16>(tmap_x, tmap_w, p, tiles, st);
    case 32: return launch_one<KIND, 32>(tmap_x, tmap_w, p, tiles, st);
    case 64: return launch_one<KIND, 64>(tmap_x, tmap_w, p, tiles, st);
    default: return launch_one<KIND, 128>(tmap_x, tmap_w, p, tiles, st);
  }
}

}  // namespace

SplitKPlan splitk_plan(int64_t T, int N, int64_t row_bytes, int sms) {
  SplitKPlan pl = {};
  const int nt = T <= 16 ? 16 : T <= 32 ? 32 : T <= 64 ? 64 : 128;
  const int64_t tiles = (T + nt - 1) / nt * ((N + kSkRows - 1) / kSkRows);
  const int k_blocks = int((row_bytes + 127) / 128);
  if (tiles > sms / 2) return pl;
  int split = 8;
  while (split > 1 && (tiles * split > 2 * sms || split > k_blocks)) split >>= 1;
  pl.nt = nt;
  pl.split = split;
  pl.tiles = int(tiles);
  pl.k_blocks = k_blocks;
  return pl;
}

cudaError_t launch_splitk(bool bf16, int nt, const void* tmap_x, const void* tmap_w,
                          const SplitKParams& p, int tiles, cudaStream_t st) {
  return bf16 ? launch_nt<kSkBF16>(nt, tmap_x, tmap_w, p, tiles, st)
              : launch_nt<kSkI8>(nt, tmap_x, tmap_w, p, tiles, st);
}

}  // namespace hq
