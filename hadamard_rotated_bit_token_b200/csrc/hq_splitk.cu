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

__device__ __forceinline__ uint4 ld_cluster_v4(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared::cluster.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr));
  return v;
}

// The split's partial sums of four weight rows from `src` on, added in rank
// order, for two tokens at a time (all 2 SPLIT loads in flight at once).
template <int KIND, int SPLIT>
__device__ __forceinline__ void join(const float* src0, const float* src1, uint4 (&sum)[2]) {
  uint4 v[2][SPLIT];
#pragma unroll
  for (int k = 0; k < SPLIT; ++k) {
    v[0][k] = ld_cluster_v4(mapa_shared(src0, uint32_t(k)));
    v[1][k] = ld_cluster_v4(mapa_shared(src1, uint32_t(k)));
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    sum[i] = v[i][0];
#pragma unroll
    for (int k = 1; k < SPLIT; ++k) {
      const uint4 w = v[i][k];
      if constexpr (KIND == kSkBF16) {
        sum[i].x = __float_as_uint(__uint_as_float(sum[i].x) + __uint_as_float(w.x));
        sum[i].y = __float_as_uint(__uint_as_float(sum[i].y) + __uint_as_float(w.y));
        sum[i].z = __float_as_uint(__uint_as_float(sum[i].z) + __uint_as_float(w.z));
        sum[i].w = __float_as_uint(__uint_as_float(sum[i].w) + __uint_as_float(w.w));
      } else {
        sum[i].x += w.x, sum[i].y += w.y, sum[i].z += w.z, sum[i].w += w.w;
      }
    }
  }
}

// Four columns from n on of row t: sums -> the epilogue -> Y.
template <int KIND>
__device__ __forceinline__ void finish4(const SplitKParams& p, const uint4& s, int t, int n) {
  f2 z[2];
  if constexpr (KIND == kSkBF16) {
    z[0] = pk(__uint_as_float(s.x), __uint_as_float(s.y));
    z[1] = pk(__uint_as_float(s.z), __uint_as_float(s.w));
    if (p.bias16) {
      const uint2 b = *reinterpret_cast<const uint2*>(p.bias16 + n);
      z[0] = add2(z[0], unpack_bf16x2(b.x));
      z[1] = add2(z[1], unpack_bf16x2(b.y));
    }
  } else {
    const float sx = p.a_scale_per_row ? p.a_scale[t] : p.a_scale[0];
    const float4 sw = *reinterpret_cast<const float4*>(p.w_scale + n);
    float4 c = p.bias ? *reinterpret_cast<const float4*>(p.bias + n) : make_float4(0, 0, 0, 0);
    f2 c0 = pk(c.x, c.y), c1 = pk(c.z, c.w);
    if (p.a_mean) {
      const float m = p.a_mean[t];
      const float4 cs = *reinterpret_cast<const float4*>(p.colsum + n);
      c0 = fma2(pk(m, m), pk(cs.x, cs.y), c0);
      c1 = fma2(pk(m, m), pk(cs.z, cs.w), c1);
    }
    z[0] = fma2(pk(__int2float_rn(int(s.x)), __int2float_rn(int(s.y))),
                mul2(pk(sx, sx), pk(sw.x, sw.y)), c0);
    z[1] = fma2(pk(__int2float_rn(int(s.z)), __int2float_rn(int(s.w))),
                mul2(pk(sx, sx), pk(sw.z, sw.w)), c1);
  }
  act_chunk(p.act, z);
  const int64_t off = int64_t(t) * p.N + n;
  if (p.gate) {
    const uint2 g = *reinterpret_cast<const uint2*>(p.gate + (t / p.gate_rows) * p.N + n);
    z[0] = mul2(z[0], unpack_bf16x2(g.x));
    z[1] = mul2(z[1], unpack_bf16x2(g.y));
  }
  if (p.residual) {
    const uint2 r = *reinterpret_cast<const uint2*>(p.residual + off);
    z[0] = add2(z[0], unpack_bf16x2(r.x));
    z[1] = add2(z[1], unpack_bf16x2(r.y));
  }
  *reinterpret_cast<uint2*>(p.Y + off) =
      make_uint2(pack_bf16x2(z[0].x, z[0].y), pack_bf16x2(z[1].x, z[1].y));
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
  auto load = [&](int kb, int stage) {
    mbar_arrive_expect_tx(&full[stage], C::STAGE_BYTES);
    tma_load_2d(sW + size_t(stage) * C::W_BYTES, &tmW, kb * 128, n0, &full[stage]);
    tma_load_2d(sX + size_t(stage) * C::X_BYTES, &tmX, kb * 128, t0, &full[stage]);
  };

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::STAGES; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    mbar_init(tfull, 1);
    *failed = 0;
    fence_mbarrier_init();
    // the first round of stages is empty: its loads go out before the other
    // warps and tensor memory are ready
    for (int kb = kb0; kb < kb1 && kb < kb0 + C::STAGES; ++kb) load(kb, kb - kb0);
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
      int stage = 0, issued = min(kb1 - kb0, C::STAGES);
      uint32_t phase = 1;
      for (int kb = kb0 + C::STAGES; kb < kb1; ++kb) {
        if (*failed || !mbar_wait(&empty[stage], phase ^ 1u, wc)) {
          *failed = 1;
          break;
        }
        load(kb, stage);
        ++issued;
        if (++stage == C::STAGES) {
          stage = 0;
          phase ^= 1u;
        }
      }
      if (*failed) {
        // the copies in flight land before the CTA can exit
        for (int i = issued > C::STAGES ? issued - C::STAGES : 0; i < issued; ++i)
          (void)mbar_wait(&full[i % C::STAGES], uint32_t(i / C::STAGES) & 1u, wc);
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
    // this CTA's share of the tokens, a warp a token, four weight rows a lane
    const int tb = NT * rank / p.split, te = NT * (rank + 1) / p.split;
    const int n = n0 + 4 * lane;
    constexpr int kWarps = kSkThreads / 32;
    for (int tt = tb + warp; tt < te && t0 + tt < p.T; tt += 2 * kWarps) {
      const int t2 = tt + kWarps < te ? tt + kWarps : tt;
      const float* s0 = part + tt * kSkRows + 4 * lane;
      const float* s1 = part + t2 * kSkRows + 4 * lane;
      uint4 sum[2];
      if (p.split == 8)
        join<KIND, 8>(s0, s1, sum);
      else if (p.split == 4)
        join<KIND, 4>(s0, s1, sum);
      else if (p.split == 2)
        join<KIND, 2>(s0, s1, sum);
      else
        join<KIND, 1>(s0, s1, sum);
      if (n < p.N) {
        finish4<KIND>(p, sum[0], t0 + tt, n);
        if (t2 != tt && t0 + t2 < p.T) finish4<KIND>(p, sum[1], t0 + t2, n);
      }
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
