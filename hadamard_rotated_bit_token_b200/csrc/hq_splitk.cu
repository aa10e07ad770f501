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
// into NT columns of tensor memory.  Every CTA owns NT / split tokens: warps
// 2..5 read the CTA's partial sums from tensor memory and write each token's
// into its owner's shared memory (distributed shared memory), and after one
// cluster barrier the owner adds the split's partial sums in rank order, applies
// the epilogue and stores.  Integer sums are exact; fp32 sums depend on the
// sizes alone.  (Owners that fetched the partial sums instead paid the remote
// latency after the barrier and a second barrier before they could leave.)
//
// Without the split a narrow layer is a few CTAs that walk all of K: 64 tokens,
// K = 4608, N = 1152 in bf16 took 23.3 us by tiles of 128 x 192 on 6 SMs, and
// 7.5 us by 9 clusters of 8 CTAs (16 tokens: 6.3 us, where one pass over the
// weights takes 1.6 us).  What is left is a chain of latencies: launch and
// tensor-memory allocation, the first TMA, the last commit, the push of the
// partial sums and the cluster's barrier.
#include <cuda.h>
#include <cuda_bf16.h>

#include <atomic>

#include "hq_act.cuh"
#include "hq_device.cuh"
#include "hq_kernels.h"

namespace hq {

namespace {

constexpr int kSkRows = 128;     // weight rows per tile (MMA M)
// producer, MMA issuer, four warps that read tensor memory; all eight join
constexpr int kSkThreads = 256;
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
  static constexpr int TMEM_COLS = NT < 32 ? 32 : NT;
  static constexpr int RECV_BYTES = NT * kSkRows * 4;  // [split][NT / split][kSkRows]
  static constexpr int CTL_BYTES = 256;
  // two CTAs an SM where that leaves three stages (deeper rings gained nothing),
  // one with 128 tokens
  static constexpr int STAGES_2 = (110 * 1024 - RECV_BYTES) / STAGE_BYTES;
  static constexpr int STAGES =
      STAGES_2 >= 3 ? STAGES_2 : (224 * 1024 - RECV_BYTES) / STAGE_BYTES;
  static constexpr size_t smem(int stages) {
    return size_t(stages) * STAGE_BYTES + RECV_BYTES + CTL_BYTES + 1024;
  }
  static_assert(X_BYTES % 1024 == 0, "stage bases stay 1024-byte aligned");
  static_assert(16 * STAGES + 32 <= CTL_BYTES, "barrier block");
};

// sum + the partial sums v, per element
template <int KIND>
__device__ __forceinline__ void add_parts(uint4& sum, const uint4& v) {
  if constexpr (KIND == kSkBF16) {
    sum.x = __float_as_uint(__uint_as_float(sum.x) + __uint_as_float(v.x));
    sum.y = __float_as_uint(__uint_as_float(sum.y) + __uint_as_float(v.y));
    sum.z = __float_as_uint(__uint_as_float(sum.z) + __uint_as_float(v.z));
    sum.w = __float_as_uint(__uint_as_float(sum.w) + __uint_as_float(v.w));
  } else {
    sum.x += v.x, sum.y += v.y, sum.z += v.z, sum.w += v.w;
  }
}

// What the epilogue needs of four columns (the same for every token), and of a
// token's four outputs; loaded before the sums they are added to are there.
struct SkCols {
  float4 sw, b, cs;
};
struct SkRow {
  float sx, m;
  uint2 gate, res;
};

template <int KIND>
__device__ __forceinline__ void load_cols(const SplitKParams& p, int n, SkCols& c) {
  c.b = c.cs = c.sw = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  if (n >= p.N) return;
  if constexpr (KIND == kSkBF16) {
    if (p.bias16) {
      const uint2 b = *reinterpret_cast<const uint2*>(p.bias16 + n);
      const f2 lo = unpack_bf16x2(b.x), hi = unpack_bf16x2(b.y);
      c.b = make_float4(lo.x, lo.y, hi.x, hi.y);
    }
  } else {
    c.sw = *reinterpret_cast<const float4*>(p.w_scale + n);
    if (p.bias) c.b = *reinterpret_cast<const float4*>(p.bias + n);
    if (p.a_mean) c.cs = *reinterpret_cast<const float4*>(p.colsum + n);
  }
}

template <int KIND>
__device__ __forceinline__ void load_row(const SplitKParams& p, int64_t t, int n, SkRow& r) {
  r.sx = r.m = 0.0f;
  r.gate = r.res = make_uint2(0, 0);
  if (t >= p.T || n >= p.N) return;
  if constexpr (KIND == kSkI8) {
    r.sx = p.a_scale_per_row ? p.a_scale[t] : p.a_scale[0];
    if (p.a_mean) r.m = p.a_mean[t];
  }
  if (p.gate) r.gate = *reinterpret_cast<const uint2*>(p.gate + (t / p.gate_rows) * p.N + n);
  if (p.residual) r.res = *reinterpret_cast<const uint2*>(p.residual + t * p.N + n);
}

// Four columns from n on of row t: sums -> the epilogue -> Y.
template <int KIND>
__device__ __forceinline__ void finish4(const SplitKParams& p, const uint4& s, const SkCols& c,
                                        const SkRow& r, int64_t t, int n) {
  f2 z[2];
  if constexpr (KIND == kSkBF16) {
    z[0] = add2(pk(__uint_as_float(s.x), __uint_as_float(s.y)), pk(c.b.x, c.b.y));
    z[1] = add2(pk(__uint_as_float(s.z), __uint_as_float(s.w)), pk(c.b.z, c.b.w));
  } else {
    const f2 sx = pk(r.sx, r.sx), m = pk(r.m, r.m);
    z[0] = fma2(pk(__int2float_rn(int(s.x)), __int2float_rn(int(s.y))),
                mul2(sx, pk(c.sw.x, c.sw.y)), fma2(m, pk(c.cs.x, c.cs.y), pk(c.b.x, c.b.y)));
    z[1] = fma2(pk(__int2float_rn(int(s.z)), __int2float_rn(int(s.w))),
                mul2(sx, pk(c.sw.z, c.sw.w)), fma2(m, pk(c.cs.z, c.cs.w), pk(c.b.z, c.b.w)));
  }
  act_chunk(p.act, z);
  if (p.gate) {
    z[0] = mul2(z[0], unpack_bf16x2(r.gate.x));
    z[1] = mul2(z[1], unpack_bf16x2(r.gate.y));
  }
  if (p.residual) {
    z[0] = add2(z[0], unpack_bf16x2(r.res.x));
    z[1] = add2(z[1], unpack_bf16x2(r.res.y));
  }
  *reinterpret_cast<uint2*>(p.Y + t * p.N + n) =
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
  const int stages = p.stages;
  uint8_t* sW = smem;
  uint8_t* sX = smem + size_t(stages) * C::W_BYTES;
  uint32_t* recv = reinterpret_cast<uint32_t*>(smem + size_t(stages) * C::STAGE_BYTES);
  uint64_t* full = reinterpret_cast<uint64_t*>(recv + C::RECV_BYTES / 4);
  uint64_t* empty = full + stages;
  uint64_t* tfull = empty + stages;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(tfull + 1);
  volatile int* failed = reinterpret_cast<volatile int*>(tmem_slot + 1);
  volatile int* issued = failed + 1;  // stages the producer has loaded

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const WaitCtl wc{p.err, p.wait_ns};
  const int rank = int(cluster_ctarank());
  const int log_own = p.log_nt - p.log_split;  // tokens per owner
  const int tile = int(blockIdx.x) >> p.log_split;
  const int tile_t = tile / p.num_n_tiles;
  const int n0 = (tile - tile_t * p.num_n_tiles) * kSkRows;
  const int t0 = tile_t * NT;
  const int kb0 = (p.k_blocks * rank) >> p.log_split;
  const int nkb = ((p.k_blocks * (rank + 1)) >> p.log_split) - kb0;

  // every CTA of the cluster has started before any writes to another
  asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
  if (warp == 0) {
    if (lane == 0) {
      for (int s = 0; s < 2 * stages + 1; ++s)  // full, empty, tfull
        mbar_init(&full[s], s == 0 && p.withhold ? 2 : 1);
      *failed = 0;
      fence_mbarrier_init();
    }
    __syncwarp();
    // the others wait for the barriers and tensor memory; this warp goes on
    asm volatile("bar.arrive 1, %0;" ::"n"(kSkThreads) : "memory");
    if (lane == 0) {
      int stage = 0;
      uint32_t phase = 0;
      int i = 0;
      for (; i < nkb; ++i) {
        if (i >= stages && !mbar_wait(&empty[stage], phase ^ 1u, wc)) {
          *failed = 1;
          break;
        }
        const int x = (kb0 + i) * 128;
        mbar_arrive_expect_tx(&full[stage], C::STAGE_BYTES);
        tma_load_2d(sW + size_t(stage) * C::W_BYTES, &tmW, x, n0, &full[stage]);
        tma_load_2d(sX + size_t(stage) * C::X_BYTES, &tmX, x, t0, &full[stage]);
        if (++stage == stages) {
          stage = 0;
          phase ^= 1u;
        }
      }
      *issued = i;
    }
  } else {
    if (warp == 1) {
      tmem_alloc(tmem_slot, C::TMEM_COLS);
      tmem_relinquish();
      tc_fence_before();
    }
    asm volatile("bar.sync 1, %0;" ::"n"(kSkThreads) : "memory");
    tc_fence_after();
  }

  // what the epilogue needs from global memory, in flight during the product:
  // a warp a token (two at a time), four weight rows a lane
  const int n = n0 + 4 * lane;
  const int own = 1 << log_own, tb = t0 + rank * own;
  constexpr int kWarps = kSkThreads / 32;
  SkCols cols;
  SkRow row[2];
  if (warp >= 2) {
    load_cols<KIND>(p, n, cols);
    load_row<KIND>(p, int64_t(tb) + warp, warp < own ? n : p.N, row[0]);
    load_row<KIND>(p, int64_t(tb) + warp + kWarps, warp + kWarps < own ? n : p.N, row[1]);
  }

  if (warp == 1) {
    const uint32_t tmem = *tmem_slot;
    const bool leader = elect_one();
    const uint64_t wd0 = sk_desc(smem_u32(sW)), xd0 = sk_desc(smem_u32(sX));
    int stage = 0;
    uint32_t phase = 0;
    for (int i = 0; i < nkb; ++i) {
      const bool got = mbar_wait(&full[stage], phase, wc);
      if (!__all_sync(0xffffffffu, got)) {
        *failed = 1;
        break;
      }
      tc_fence_after();
      if (leader) {
        const uint64_t wd = wd0 + uint64_t(stage) * (C::W_BYTES >> 4);
        const uint64_t xd = xd0 + uint64_t(stage) * (C::X_BYTES >> 4);
#pragma unroll
        for (int k = 0; k < 4; ++k) {  // 32 bytes along K inside the swizzle row
          if constexpr (KIND == kSkBF16)
            mma_bf16(tmem, wd + uint64_t(2 * k), xd + uint64_t(2 * k), sk_idesc<KIND>(NT),
                     (i > 0 || k > 0) ? 1u : 0u);
          else
            mma_i8(tmem, wd + uint64_t(2 * k), xd + uint64_t(2 * k), sk_idesc<KIND>(NT),
                   (i > 0 || k > 0) ? 1u : 0u);
        }
        if (i + stages < nkb) mma_commit(&empty[stage]);
      }
      __syncwarp();
      if (++stage == stages) {
        stage = 0;
        phase ^= 1u;
      }
    }
    if (leader) mma_commit(tfull);  // every MMA issued has completed
    __syncwarp();
  }
  __syncwarp();
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
  if (warp >= 1 && warp < 6) {
    const bool got = mbar_wait(tfull, 0, wc);
    if (__all_sync(0xffffffffu, got) && warp >= 2 && !*failed) {
      tc_fence_after();
      // lane quarter warp % 4 of tensor memory: weight rows 32 q + lane
      const int q = warp & 3;
      const uint32_t* dst = recv + (rank << log_own) * kSkRows + q * 32 + lane;
#pragma unroll
      for (int c = 0; c < NT; c += 32) {
        uint32_t r[32];
        tmem_ld_32x32b_x32(*tmem_slot + (uint32_t(q * 32) << 16) + uint32_t(c), r);
        tmem_wait_ld();
#pragma unroll
        for (int i = 0; i < 32; ++i) {
          const int t = c + i;
          if (t < NT && t0 + t < p.T)
            st_shared_cluster_u32(
                mapa_shared(dst + (t & (own - 1)) * kSkRows, uint32_t(t >> log_own)), r[i]);
        }
      }
    } else if (!got) {
      *failed = 1;
    }
  }
  if (warp < 2) {
    load_cols<KIND>(p, n, cols);
    load_row<KIND>(p, int64_t(tb) + warp, warp < own ? n : p.N, row[0]);
    load_row<KIND>(p, int64_t(tb) + warp + kWarps, warp + kWarps < own ? n : p.N, row[1]);
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // every CTA's partial sums are with their owners

  // After a give-up, whichever wait it was, the copies in flight land and the
  // MMAs issued complete before the CTA can exit.
  if (*failed && threadIdx.x == 0) {
    const int i = *issued;
    for (int j = i > stages ? i - stages : 0; j < i; ++j)
      (void)mbar_wait(&full[j % stages], uint32_t(j / stages) & 1u, wc);
    (void)mbar_wait(tfull, 0, wc);
  }
  if (!*failed && n < p.N) {
    const uint4* src = reinterpret_cast<const uint4*>(recv) + lane;
    for (int i = warp; i < own && tb + i < p.T; i += 2 * kWarps) {
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int tt = i + j * kWarps;
        if (tt < own && tb + tt < p.T) {
          uint4 sum = src[tt * (kSkRows / 4)];
#pragma unroll 4
          for (int k = 1; k < (1 << p.log_split); ++k)
            add_parts<KIND>(sum, src[((k << log_own) + tt) * (kSkRows / 4)]);
          finish4<KIND>(p, sum, cols, row[j], int64_t(tb) + tt, n);
        }
        load_row<KIND>(p, int64_t(tb) + tt + 2 * kWarps, tt + 2 * kWarps < own ? n : p.N, row[j]);
      }
    }
  }
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(*tmem_slot, C::TMEM_COLS);
  }
}

namespace {

template <int KIND, int NT>
cudaError_t launch_one(const void* tmap_x, const void* tmap_w, SplitKParams p, int tiles,
                       cudaStream_t st) {
  using C = SkCfg<NT>;
  const void* fn = (const void*)splitk_kernel<KIND, NT>;
  static std::atomic<unsigned long long> done{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const unsigned long long bit = 1ull << (dev & 63);
  if (!(done.load(std::memory_order_relaxed) & bit)) {
    e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             int(C::smem(C::STAGES)));
    if (e != cudaSuccess) return e;
    done.fetch_or(bit, std::memory_order_relaxed);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(tiles) << p.log_split);
  cfg.blockDim = dim3(kSkThreads);
  const int split = 1 << p.log_split;
  const int blocks = (p.k_blocks + split - 1) / split;
  p.stages = blocks > C::STAGES ? C::STAGES : blocks;
  p.log_nt = NT == 16 ? 4 : NT == 32 ? 5 : NT == 64 ? 6 : 7;
  cfg.dynamicSmemBytes = C::smem(p.stages);
  cfg.stream = st;
  cudaLaunchAttribute a[1];
  a[0].id = cudaLaunchAttributeClusterDimension;
  a[0].val.clusterDim.x = 1u << p.log_split;
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

// The tile and split of the least modelled time, in microseconds, fitted to
// sweeps of 4 to 512 tokens over layers of 256 to 4608 inputs and 1152 to 16384
// outputs in both types: a launch and its barriers, 0.2 a K block (no faster
// than the weights arrive), 0.03 a token for the exchange and 0.055 for each that
// a CTA owns; stretched once the grid passes one CTA an SM.
SplitKPlan splitk_plan(int64_t T, int N, int64_t row_bytes, int sms) {
  SplitKPlan best = {};
  best.us = 1e30;
  const int k_blocks = int((row_bytes + 127) / 128);
  const double arrive = weights_us(N, row_bytes);
  for (int nt : {16, 32, 64, 128}) {
    if (nt > 16 && nt >= 2 * T) break;
    const int64_t tiles = splitk_tiles(T, N, nt);
    for (int ls = 0; ls <= 3 && (1 << ls) <= k_blocks; ++ls) {
      if ((tiles << ls) > 4 * int64_t(sms)) break;
      double f = double(tiles << ls) / sms;
      if (f < 1.0) f = 1.0;
      // one CTA an SM, and clusters of four or eight leave some SMs without one:
      // whole waves
      const int64_t at_once = ls >= 2 ? int64_t(sms) * 6 / 7 : sms;
      if (nt == 128) f = double(((tiles << ls) + at_once - 1) / at_once);
      double product = 0.2 * ((k_blocks >> ls) + 1) * f;
      if (product < arrive) product = arrive;
      const double us = 3.9 + product + (0.03 * nt + 0.055 * (nt >> ls)) * f;
      if (us < best.us) best = SplitKPlan{us, nt, ls};
    }
  }
  return best;
}

cudaError_t launch_splitk(bool bf16, int nt, const void* tmap_x, const void* tmap_w,
                          const SplitKParams& p, int tiles, cudaStream_t st) {
  return bf16 ? launch_nt<kSkBF16>(nt, tmap_x, tmap_w, p, tiles, st)
              : launch_nt<kSkI8>(nt, tmap_x, tmap_w, p, tiles, st);
}

}  // namespace hq
