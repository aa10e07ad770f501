// hq_norm.cu -- group norm with an activation over channels-last tensors.
//
//   y = act((x - mean) / sqrt(var + eps) * gamma_c + beta_c)
//
// with mean and variance over the S pixels and C / G channels of an image's
// group.  Two launches: gn_stats_kernel leaves each row chunk's (mean, sum of
// squared deviations) per group in the workspace, gn_apply_kernel merges the
// chunks' statistics and normalizes.
//
// Statistics never subtract large sums: a thread accumulates deviations from
// its own first value of the channel, turns them into (mean, M2), and parts i
// of n_i values merge as  mean = mean_0 + sum n_i (mean_i - mean_0) / n,
// M2 = sum M2_i + n_i (mean_i - mean)^2  (equal values: mean exactly theirs).
#include <cuda_bf16.h>

#include "hq_act.cuh"
#include "hq_device.cuh"
#include "hq_kernels.h"

namespace hq {

namespace {

constexpr int kGnThreads = 256;

template <int VEC>
struct Vec;
template <>
struct Vec<8> { typedef uint4 T; };
template <>
struct Vec<4> { typedef uint2 T; };
template <>
struct Vec<2> { typedef uint32_t T; };
template <>
struct Vec<1> { typedef uint16_t T; };

template <int VEC>
__device__ __forceinline__ void load_vec(const uint16_t* p, float (&v)[VEC]) {
  const typename Vec<VEC>::T raw = *reinterpret_cast<const typename Vec<VEC>::T*>(p);
  const uint16_t* h = reinterpret_cast<const uint16_t*>(&raw);
#pragma unroll
  for (int i = 0; i < VEC; ++i) v[i] = __uint_as_float(uint32_t(h[i]) << 16);
}

template <int VEC>
__device__ __forceinline__ void store_vec(uint16_t* p, const float (&v)[VEC]) {
  typename Vec<VEC>::T raw;
  __nv_bfloat16* h = reinterpret_cast<__nv_bfloat16*>(&raw);
#pragma unroll
  for (int i = 0; i < VEC; ++i) h[i] = __float2bfloat16_rn(v[i]);
  *reinterpret_cast<typename Vec<VEC>::T*>(p) = raw;
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

}  // namespace

// One CTA: a chunk of rows of one image.  Threads sit rp x cv over rows
// and channel vectors; the per-channel parts of the rp threads merge in shared
// memory, then a warp per group merges the group's channels.
template <int VEC>
__global__ void __launch_bounds__(kGnThreads) gn_stats_kernel(const GnParams p) {
  extern __shared__ float2 sm[];
  float2* chan = sm;         // [C] (mean, M2) over the chunk's rows
  float2* part = sm + p.C;   // [kGnThreads * VEC] per thread and channel
  const int64_t b = blockIdx.x / unsigned(p.P);
  const int chunk = int(blockIdx.x % unsigned(p.P));
  const int64_t r0 = int64_t(chunk) * p.rows_p;
  const int64_t r1 = r0 + p.rows_p < p.S ? r0 + p.rows_p : p.S;
  const int rows = int(r1 - r0);
  const int CV = p.C / VEC;
  const uint16_t* base = p.X + (b * p.S + r0) * p.C;
  for (int v0 = 0; v0 < CV; v0 += kGnThreads) {
    const int nv = CV - v0 < kGnThreads ? CV - v0 : kGnThreads;  // vectors in this pass
    const int RP = kGnThreads / nv;                              // rows side by side
    const int rp = threadIdx.x / nv, cv = threadIdx.x % nv;
    if (rp < RP && rp < rows) {
      const uint16_t* x = base + int64_t(rp) * p.C + (v0 + cv) * VEC;
      float piv[VEC], s1[VEC], s2[VEC];
      load_vec<VEC>(x, piv);
#pragma unroll
      for (int i = 0; i < VEC; ++i) s1[i] = s2[i] = 0.0f;
      int n = 0;
      for (int r = rp; r < rows; r += RP, x += int64_t(RP) * p.C, ++n) {
        float v[VEC];
        load_vec<VEC>(x, v);
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
          const float d = v[i] - piv[i];
          s1[i] += d;
          s2[i] = fmaf(d, d, s2[i]);
        }
      }
      const float inv = 1.0f / float(n);
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        const float m = s1[i] * inv;
        part[rp * (nv * VEC) + cv * VEC + i] =
            make_float2(piv[i] + m, fmaxf(fmaf(-s1[i], m, s2[i]), 0.0f));
      }
    }
    __syncthreads();
    const int used = RP < rows ? RP : rows;
    for (int c = threadIdx.x; c < nv * VEC; c += kGnThreads) {
      // rows of thread rp: ceil((rows - rp) / RP)
      const float ref = part[c].x;
      float mean = 0.0f;
      for (int i = 1; i < used; ++i)
        mean = fmaf(float((rows - i + RP - 1) / RP), part[i * (nv * VEC) + c].x - ref, mean);
      mean = ref + mean / float(rows);
      float m2 = 0.0f;
      for (int i = 0; i < used; ++i) {
        const float2 q = part[i * (nv * VEC) + c];
        const float d = q.x - mean;
        m2 += fmaf(float((rows - i + RP - 1) / RP) * d, d, q.y);
      }
      chan[v0 * VEC + c] = make_float2(mean, m2);
    }
    __syncthreads();
  }
  const int cpg = p.C / p.G;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int g = warp; g < p.G; g += kGnThreads / 32) {
    const float ref = chan[g * cpg].x;
    float mean = 0.0f;
    for (int c = lane; c < cpg; c += 32) mean += chan[g * cpg + c].x - ref;
    mean = ref + warp_sum(mean) / float(cpg);
    float m2 = 0.0f;
    for (int c = lane; c < cpg; c += 32) {
      const float2 q = chan[g * cpg + c];
      const float d = q.x - mean;
      m2 += fmaf(float(rows) * d, d, q.y);
    }
    m2 = warp_sum(m2);
    if (lane == 0) p.part[(b * p.P + chunk) * p.G + g] = make_float2(mean, m2);
  }
}

// One CTA: rows of one image, normalized with the merged statistics.
template <int VEC>
__global__ void __launch_bounds__(kGnThreads) gn_apply_kernel(const GnParams p, int chunks,
                                                             int64_t rows_a) {
  extern __shared__ float2 stat[];  // [G] (mean, 1 / sqrt(var + eps))
  const int64_t b = blockIdx.x / unsigned(chunks);
  const int cpg = p.C / p.G;
  for (int g = threadIdx.x; g < p.G; g += kGnThreads) {
    const float2* q = p.part + b * p.P * p.G + g;
    auto rows_of = [&](int i) {
      const int64_t left = p.S - int64_t(i) * p.rows_p;
      return float(left < p.rows_p ? left : p.rows_p);
    };
    const float ref = q[0].x;
    float mean = 0.0f;
    for (int i = 1; i < p.P; ++i) mean = fmaf(rows_of(i), q[int64_t(i) * p.G].x - ref, mean);
    mean = ref + mean / float(p.S);
    float m2 = 0.0f;
    for (int i = 0; i < p.P; ++i) {
      const float2 v = q[int64_t(i) * p.G];
      const float d = v.x - mean;
      m2 += fmaf(rows_of(i) * float(cpg) * d, d, v.y);
    }
    const float var = m2 / (float(p.S) * float(cpg));
    stat[g] = make_float2(mean, 1.0f / sqrtf(var + p.eps));
  }
  __syncthreads();
  const int64_t r0 = int64_t(blockIdx.x % unsigned(chunks)) * rows_a;
  const int64_t r1 = r0 + rows_a < p.S ? r0 + rows_a : p.S;
  const int CV = p.C / VEC;
  for (int v0 = 0; v0 < CV; v0 += kGnThreads) {
    const int nv = CV - v0 < kGnThreads ? CV - v0 : kGnThreads;
    const int RP = kGnThreads / nv;
    const int rp = threadIdx.x / nv, cv = threadIdx.x % nv;
    if (rp >= RP) continue;
    const int c0 = (v0 + cv) * VEC;
    float mean[VEC], a[VEC], be[VEC];
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
      const float2 s = stat[(c0 + i) / cpg];
      mean[i] = s.x;
      a[i] = s.y * (p.gamma ? __uint_as_float(uint32_t(p.gamma[c0 + i]) << 16) : 1.0f);
      be[i] = p.beta ? __uint_as_float(uint32_t(p.beta[c0 + i]) << 16) : 0.0f;
    }
    for (int64_t r = r0 + rp; r < r1; r += RP) {
      const int64_t off = (b * p.S + r) * p.C + c0;
      float v[VEC];
      load_vec<VEC>(p.X + off, v);
      constexpr int NP = (VEC + 1) / 2;
      f2 z[NP];
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        const float y = fmaf(v[i] - mean[i], a[i], be[i]);
        if (i & 1) z[i / 2].y = y; else z[i / 2].x = y;
      }
      if constexpr (VEC == 1) z[0].y = 0.0f;
      act_chunk<NP>(p.act, z);
#pragma unroll
      for (int i = 0; i < VEC; ++i) v[i] = (i & 1) ? z[i / 2].y : z[i / 2].x;
      store_vec<VEC>(p.Y + off, v);
    }
  }
}

// Row chunks per image: enough CTAs for two a multiprocessor, at most 64.
int gn_chunks(int64_t B, int64_t S, int C, int sms) {
  (void)C;
  int64_t want = (2 * int64_t(sms) + B - 1) / B;
  if (want > 64) want = 64;
  if (want > S) want = S;
  if (want < 1) want = 1;
  const int64_t rows = (S + want - 1) / want;
  return int((S + rows - 1) / rows);
}

template <int VEC>
static cudaError_t launch_gn(const GnParams& p, int sms, cudaStream_t st) {
  const size_t smem_s = sizeof(float2) * (size_t(p.C) + kGnThreads * VEC);
  const size_t smem_a = sizeof(float2) * size_t(p.G);
  cudaError_t e = cudaFuncSetAttribute(gn_stats_kernel<VEC>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, 96 * 1024);
  if (e != cudaSuccess) return e;
  e = cudaFuncSetAttribute(gn_apply_kernel<VEC>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           96 * 1024);
  if (e != cudaSuccess) return e;
  gn_stats_kernel<VEC><<<unsigned(p.P * p.B), kGnThreads, smem_s, st>>>(p);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  int64_t chunks = (8 * int64_t(sms) + p.B - 1) / p.B;
  if (chunks > p.S) chunks = p.S;
  const int64_t rows = (p.S + chunks - 1) / chunks;
  chunks = (p.S + rows - 1) / rows;
  gn_apply_kernel<VEC><<<unsigned(chunks * p.B), kGnThreads, smem_a, st>>>(p, int(chunks), rows);
  return cudaGetLastError();
}

cudaError_t launch_group_norm(const GnParams& p, int sms, cudaStream_t st) {
  if (p.C % 8 == 0) return launch_gn<8>(p, sms, st);
  if (p.C % 4 == 0) return launch_gn<4>(p, sms, st);
  if (p.C % 2 == 0) return launch_gn<2>(p, sms, st);
  return launch_gn<1>(p, sms, st);
}

}  // namespace hq
