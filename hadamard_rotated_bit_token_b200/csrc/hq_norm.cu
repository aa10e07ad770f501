// hq_norm.cu -- group norm with an activation over channels-last tensors.
//
//   y = act((x - mean) / sqrt(var + eps) * gamma_c + beta_c)
//
// with mean and variance over the S pixels and C / G channels of an image's
// group.  A small tensor is one launch, gn_small_kernel, in registers.  Others
// are two: gn_stats_kernel leaves (mean, M2 = sum of squared
// deviations) of every row chunk and group in the workspace; gn_apply_kernel,
// launched as its programmatic dependent (it starts while the first drains,
// loads its first rows, and waits), merges the chunks' statistics, normalizes
// and writes.  X is read twice, the second time from L2 as far as the tensor
// fits there.
//
// Statistics never subtract large sums.  Parts i of n_i values with mean m_i
// and M2 q_i merge around the first part's mean m_0:
//   s1 = sum n_i (m_i - m_0),  s2 = sum q_i + n_i (m_i - m_0)^2,
//   mean = m_0 + s1 / n,  M2 = s2 - s1^2 / n.
// Part 0 itself adds n_0 (m_0 - mean)^2 to M2, so (m_0 - mean)^2 n <= M2 n / n_0
// and the subtraction costs at most a factor n / n_0, the number of parts,
// whatever the data.  A thread's values of one channel merge the same way
// around the first of them, and around their mean so far after every 128 (a
// first value far from thousands of equal ones: their squares' roundings add up
// one way, and the factor makes 24 % of the variance of them at 4047 values, 3e-5
// so).  Orders depend on sizes alone; equal values give exactly their mean and
// M2 = 0.
//
// Why two passes of one CTA an SM, where the tensor does not fit the registers:
// keeping a few groups at a time resident over a cluster (X read once) was tried
// first and took 59 us for 16 x 4096 x 320 and 184 us for 262144 x 128: every
// unit of work paid a load, a cluster barrier and a store one after the other.
// Streaming takes 26.0 us (42 MB read, read again mostly from L2, 42 MB written:
// 3.2 TB/s of X read once and Y written) and 38.0 us (67 MB in, 67 MB out: 3.5
// TB/s).  Neither pass is at a limit of the hardware: the statistics read 42 MB in
// 12.7 us (3.3 TB/s, half of what a copy reaches) with 39 % of the issue slots used,
// the normalization (about 120 instructions for 8 channels with silu) has issue
// slots and special functions half busy.  Both wait for their own 16 warps an SM,
// whose loads in flight and dependent instructions do not cover the latencies.
// Two CTAs an SM, or one, two or three rows a batch, made the second slower (28 to
// 30 us).
#include <cuda_bf16.h>

#include <atomic>
#include <cmath>

#include "hq_act.cuh"
#include "hq_device.cuh"
#include "hq_kernels.h"

namespace hq {

namespace {

constexpr int kGnThreads = 512;
// A thread's sums move to the mean so far after this many values of a channel.
constexpr int kRecenter = 128;
// Per-thread parts: value i of thread t at part[i * kPartLd + t], so a warp
// stores without bank conflicts (and reads nearly so: the odd pitch).
constexpr int kPartLd = kGnThreads + 1;

// VEC bf16 values of consecutive channels, loaded at once.
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
__device__ __forceinline__ void unpack_vec(const typename Vec<VEC>::T& raw, float (&v)[VEC]) {
  if constexpr (VEC == 1) {
    v[0] = __uint_as_float(uint32_t(raw) << 16);
  } else {
    const uint32_t* w = reinterpret_cast<const uint32_t*>(&raw);
#pragma unroll
    for (int i = 0; i < VEC / 2; ++i) {
      const f2 p = unpack_bf16x2(w[i]);
      v[2 * i] = p.x;
      v[2 * i + 1] = p.y;
    }
  }
}

// A thread's running sums for VEC channels around each channel's first value.
template <int VEC>
struct ThreadStats {
  float piv[VEC], s1[VEC], s2[VEC];
  __device__ __forceinline__ void start(const typename Vec<VEC>::T& raw) {
    unpack_vec<VEC>(raw, piv);
#pragma unroll
    for (int i = 0; i < VEC; ++i) s1[i] = s2[i] = 0.0f;
  }
  __device__ __forceinline__ void add(const typename Vec<VEC>::T& raw) {
    float v[VEC];
    unpack_vec<VEC>(raw, v);
    if constexpr (VEC == 1) {
      const float d = v[0] - piv[0];
      s1[0] += d;
      s2[0] = fmaf(d, d, s2[0]);
    } else {
#pragma unroll
      for (int i = 0; i < VEC; i += 2) {
        const f2 d = sub2(pk(v[i], v[i + 1]), pk(piv[i], piv[i + 1]));
        const f2 a = add2(pk(s1[i], s1[i + 1]), d);
        const f2 b = fma2(d, d, pk(s2[i], s2[i + 1]));
        s1[i] = a.x, s1[i + 1] = a.y;
        s2[i] = b.x, s2[i + 1] = b.y;
      }
    }
  }
  // The same sums of n values around their mean instead (or next to it: delta is
  // what the addition to the pivot made of it).
  __device__ __forceinline__ void recenter(int n) {
    const float fn = float(n), inv = rcp_approx(fn);
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
      const float to = fmaf(s1[i], inv, piv[i]), delta = to - piv[i];
      s2[i] = fmaf(-delta, fmaf(-fn, delta, 2.0f * s1[i]), s2[i]);
      s1[i] = fmaf(-fn, delta, s1[i]);
      piv[i] = to;
    }
  }
  // (mean, M2) of n values a channel -> this thread's column of `part`
  __device__ __forceinline__ void finish(int n, float2* part) const {
    const float inv = rcp_approx(float(n));
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
      const float m = s1[i] * inv;
      part[i * kPartLd + threadIdx.x] = make_float2(piv[i] + m, s2[i] - s1[i] * m);
    }
  }
};

// Merging around `ref`: add() parts, reduce the two sums, finish().
struct Merge {
  float ref, s1, s2;
  __device__ __forceinline__ void add(float n, float2 part) {
    const float d = part.x - ref;
    s1 = fmaf(n, d, s1);
    s2 += fmaf(n * d, d, part.y);
  }
  __device__ __forceinline__ float2 finish(float inv_n) const {
    const float m = s1 * inv_n;
    return make_float2(ref + m, s2 - s1 * m);
  }
};

__device__ __forceinline__ float2 mean_rstd(float2 stat, float inv_n, float eps) {
  // the rounding of M2's subtraction can leave a tiny negative value
  const float var = stat.y * inv_n;
  // squares that overflowed: rsqrt(infinity) = 0 would give beta without a trace
  const float none = __int_as_float(0x7FFFFFFF);
  return make_float2(stat.x, var < INFINITY ? rsqrtf((var < 0.0f ? 0.0f : var) + eps) : none);
}

// x / d for x < 2^16, with magic = ceil(2^32 / d) (0 for d = 1)
__device__ __forceinline__ int div_small(int x, unsigned magic) {
  return magic ? int(__umulhi(unsigned(x), magic)) : x;
}

__device__ __forceinline__ float bf16_at(const uint16_t* p, int i, float none) {
  return p ? __uint_as_float(uint32_t(p[i]) << 16) : none;
}

// The normalization of VEC consecutive channels, and the activation.
// Coefficients of a channel: mean, a = rstd gamma, beta.
template <int VEC>
struct Normalize {
  float mean[VEC], a[VEC], b[VEC];
  // coef: [3][ld] in shared memory, this thread's channels from c on
  __device__ __forceinline__ void load(const float* coef, int ld, int c) {
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
      mean[i] = coef[c + i];
      a[i] = coef[ld + c + i];
      b[i] = coef[2 * ld + c + i];
    }
  }
  template <int ACT>
  __device__ __forceinline__ typename Vec<VEC>::T apply(const typename Vec<VEC>::T& raw) const {
    float v[VEC];
    unpack_vec<VEC>(raw, v);
    constexpr int NP = (VEC + 1) / 2;
    f2 z[NP];
    if constexpr (VEC == 1) {
      z[0] = pk(fmaf(v[0] - mean[0], a[0], b[0]), 0.0f);
    } else {
#pragma unroll
      for (int i = 0; i < NP; ++i)
        z[i] = fma2(sub2(pk(v[2 * i], v[2 * i + 1]), pk(mean[2 * i], mean[2 * i + 1])),
                    pk(a[2 * i], a[2 * i + 1]), pk(b[2 * i], b[2 * i + 1]));
    }
#pragma unroll
    for (int i = 0; i < NP; ++i) z[i] = act_one<ACT>(z[i]);
    typename Vec<VEC>::T out;
    if constexpr (VEC == 1) {
      out = uint16_t(pack_bf16x2(z[0].x, 0.0f) & 0xFFFFu);
    } else {
      uint32_t* w = reinterpret_cast<uint32_t*>(&out);
#pragma unroll
      for (int i = 0; i < NP; ++i) w[i] = pack_bf16x2(z[i].x, z[i].y);
    }
    return out;
  }
};

// The previous kernel of the stream has finished and its writes are visible.
__device__ __forceinline__ void wait_for_previous_kernel() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
}
// The next kernel of the stream may start once every CTA has come here.
__device__ __forceinline__ void let_next_kernel_start() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// The CTA's per-thread parts -> (mean, M2) of gs groups in out[0 .. gs).
// Thread t = rp * nv + cv (rp < used) holds VEC of the M = nv * VEC channels,
// with w + 1 values a channel where rp < rem and w elsewhere; channel c has
// v_hi values in all where c < vsplit, else v_lo; a group has cpg = M / gs
// channels.  kk threads a channel, then L lanes a group (p.kk, p.lanes; both
// chosen on the host).  sums: [max(kGnThreads, M)] scratch.  All threads call
// it; the parts are synchronized on entry, out is not on exit.
template <int VEC>
__device__ __forceinline__ void block_group_stats(const GnParams& p, const float2* part,
                                                  float2* sums, int used, int nv, int cpg,
                                                  int gs, float inv_n, int rem, float w,
                                                  int vsplit, float v_hi, float v_lo,
                                                  float2* out) {
  const int M = nv * VEC;
  const int k = p.kk == 1 ? 0 : div_small(int(threadIdx.x), p.magic_m);
  if (k < p.kk) {
    for (int c = int(threadIdx.x) - k * M; c < M; c += kGnThreads) {
      const float2* q = part + (c % VEC) * kPartLd + c / VEC;
      Merge m{q[0].x, 0.0f, 0.0f};
      const int stride = p.kk * nv;
      q += k * nv;
#pragma unroll 4
      for (int rp = k; rp < used; rp += p.kk, q += stride) m.add(rp < rem ? w + 1.0f : w, *q);
      sums[k * M + c] = make_float2(m.s1, m.s2);
    }
  }
  __syncthreads();
  const int L = p.lanes;
  const int l = int(threadIdx.x) & (L - 1);
  const float i_hi = rcp_approx(v_hi), i_lo = v_lo > 0.0f ? rcp_approx(v_lo) : 0.0f;
  const int per = kGnThreads >> p.log_lanes;  // groups at a time
  for (int g0 = 0; g0 < gs; g0 += per) {
    const int g = g0 + (int(threadIdx.x) >> p.log_lanes);
    const int cg = min(g, gs - 1) * cpg;
    Merge m{part[(cg % VEC) * kPartLd + cg / VEC].x, 0.0f, 0.0f};
    for (int c = cg + l; c < cg + cpg; c += L) {
      float s1 = 0.0f, s2 = 0.0f;
      for (int j = 0; j < p.kk; ++j) {
        const float2 v = sums[j * M + c];
        s1 += v.x;
        s2 += v.y;
      }
      const bool hi = c < vsplit;
      const float mc = s1 * (hi ? i_hi : i_lo);
      m.add(hi ? v_hi : v_lo,
            make_float2(part[(c % VEC) * kPartLd + c / VEC].x + mc, s2 - s1 * mc));
    }
    for (int o = L >> 1; o > 0; o >>= 1) {
      m.s1 += __shfl_xor_sync(0xffffffffu, m.s1, o);
      m.s2 += __shfl_xor_sync(0xffffffffu, m.s2, o);
    }
    if (l == 0 && g < gs) out[g] = m.finish(inv_n);
  }
}

}  // namespace

// The grid is (P, B) with images beyond 65535 along z.
__device__ __forceinline__ int64_t image_of_block() {
  return int64_t(blockIdx.z) * 65535 + blockIdx.y;
}

// One CTA: a chunk of rows of one image.  Thread rp * nv + cv walks rows rp,
// rp + RP, ... of vector column cv with eight to sixteen loads in flight.
template <int VEC>
__global__ void __launch_bounds__(kGnThreads, 1) gn_stats_kernel(const GnParams p) {
  extern __shared__ float2 sm[];
  float2* part = sm;                   // [VEC][kPartLd]
  float2* sums = sm + VEC * kPartLd;   // [max(kGnThreads, channels of a pass)]
  let_next_kernel_start();
  const int64_t b = image_of_block();
  if (b >= p.B) return;
  const int chunk = int(blockIdx.x);
  const bool last = chunk == p.P - 1;
  const int rows = last ? p.rows_last : p.rows_p;
  const float inv_n = last ? p.inv_n_last : p.inv_n_full;
  const uint16_t* base = p.X + (b * p.S + int64_t(chunk) * p.rows_p) * p.C;
  float2* outp = p.part + (b * p.P + chunk) * p.G;
  typedef typename Vec<VEC>::T V;
  const int nv = p.nv, RP = p.RP;
  // passes over slices of p.gs whole groups, at most kGnThreads vectors a row;
  // a single group may be wider: its row is then walked by all threads
  for (int g1 = 0; g1 < p.G; g1 += p.gs) {
    // (the last pass starts early enough to be a whole one: the groups it shares
    // with the one before come out the same)
    const int g0 = min(g1, p.G - p.gs);
    const uint16_t* xs = base + g0 * p.cpg;
    if (nv <= kGnThreads) {
      const int rp = div_small(int(threadIdx.x), p.magic_nv), cv = int(threadIdx.x) - rp * nv;
      const int q = last ? p.q_last : p.q_full, rem = rows - q * RP;
      if (rp < RP && rp < rows) {
        const int step = RP * p.C;
        const uint16_t* x = xs + rp * p.C + cv * VEC;
        const int cnt = rp < rem ? q + 1 : q;
        // batches of U rows, the next batch's loads out before this one is added
        constexpr int U = 8;
        V raw[U];
#pragma unroll
        for (int j = 0; j < U; ++j)
          if (j < cnt) raw[j] = *reinterpret_cast<const V*>(x + j * step);
        ThreadStats<VEC> ts;
        ts.start(raw[0]);
        int left = cnt;
        while (left >= U) {
          V cur[U];
#pragma unroll
          for (int j = 0; j < U; ++j) cur[j] = raw[j];
          x += U * step;
          left -= U;
          if (left >= U) {
#pragma unroll
            for (int j = 0; j < U; ++j) raw[j] = *reinterpret_cast<const V*>(x + j * step);
          } else {
#pragma unroll
            for (int j = 0; j < U - 1; ++j)
              if (j < left) raw[j] = *reinterpret_cast<const V*>(x + j * step);
          }
#pragma unroll
          for (int j = 0; j < U; ++j) ts.add(cur[j]);
          if ((cnt - left) % kRecenter == 0) ts.recenter(cnt - left);
        }
#pragma unroll
        for (int j = 0; j < U - 1; ++j)
          if (j < left) ts.add(raw[j]);
        ts.finish(cnt, part);
      }
      __syncthreads();
      block_group_stats<VEC>(p, part, sums, min(RP, rows), nv, p.cpg, p.gs, inv_n, rem, float(q),
                             nv * VEC, float(rows), 0.0f, outp + g0);
    } else {
      ThreadStats<VEC> ts;
      ts.start(*reinterpret_cast<const V*>(xs + threadIdx.x * VEC));
      const int q = nv / kGnThreads, rem = nv % kGnThreads;
      const int each = int(threadIdx.x) < rem ? q + 1 : q;  // vectors of a row
      int since = 0;
      for (int r = 0; r < rows; ++r, xs += p.C) {
        for (int cv = threadIdx.x; cv < nv; cv += kGnThreads)
          ts.add(*reinterpret_cast<const V*>(xs + cv * VEC));
        if ((since += each) >= kRecenter) {
          ts.recenter((r + 1) * each);
          since = 0;
        }
      }
      ts.finish(rows * each, part);
      __syncthreads();
      // as one row of kGnThreads vectors, each with the values of its thread
      block_group_stats<VEC>(p, part, sums, 1, kGnThreads, kGnThreads * VEC, 1, inv_n, 0, 0.0f,
                             rem * VEC, float(rows) * float(q + 1), float(rows) * float(q),
                             outp + g0);
    }
    if (g1 + p.gs < p.G) __syncthreads();
  }
}

// One CTA: a chunk of rows of one image, normalized with the merged
// statistics.  Chunks run from the end, whose rows the statistics read last.
template <int VEC>
__global__ void __launch_bounds__(kGnThreads, 1) gn_apply_kernel(const GnParams p) {
  extern __shared__ float2 sm[];
  float2* stat = sm;                                 // [G] (mean, 1 / sqrt(var + eps))
  float* coef = reinterpret_cast<float*>(sm + p.G);  // [3][C]
  float2* sums = reinterpret_cast<float2*>(coef + 3 * p.C + (p.C & 1));  // [kGnThreads]
  const int64_t b = p.B - 1 - image_of_block();
  if (b < 0) return;
  const int chunk = p.P - 1 - int(blockIdx.x);
  const int rows = chunk == p.P - 1 ? p.rows_last : p.rows_p;
  const int64_t base = (b * p.S + int64_t(chunk) * p.rows_p) * p.C;
  const int CV = p.C / VEC;
  typedef typename Vec<VEC>::T V;
  // the first vector column's first rows and this thread's first channel's
  // parameters, which do not depend on the statistics
  constexpr int U = 4;
  const int nva = p.nva, RPa = p.RPa;
  const int rp = div_small(int(threadIdx.x), p.magic_nva), cv = int(threadIdx.x) - rp * nva;
  const int step = RPa * p.C;
  const uint16_t* x = p.X + base + rp * p.C + cv * VEC;
  // rows of this thread
  const int q = chunk == p.P - 1 ? p.qa_last : p.qa_full;
  const int cnt = rp < rows - q * RPa ? q + 1 : q;
  V raw[U];
  if (rp < RPa) {
#pragma unroll
    for (int j = 0; j < U; ++j)
      if (j < cnt) raw[j] = *reinterpret_cast<const V*>(x + j * step);
  }
  float ga = 1.0f, be = 0.0f;
  if (int(threadIdx.x) < p.C) {
    ga = bf16_at(p.gamma, int(threadIdx.x), 1.0f);
    be = bf16_at(p.beta, int(threadIdx.x), 0.0f);
  }
  wait_for_previous_kernel();
  {
    // ka threads a group share its P parts; thread k * G + g reads parts k,
    // k + ka, ... of group g, neighbours neighbouring groups
    const float2* parts = p.part + b * p.P * p.G;
    const int k = p.ka == 1 ? 0 : div_small(int(threadIdx.x), p.magic_g);
    if (k < p.ka) {
      for (int g = int(threadIdx.x) - k * p.G; g < p.G; g += kGnThreads) {
        Merge m{parts[g].x, 0.0f, 0.0f};
        for (int i0 = k; i0 < p.P; i0 += 10 * p.ka) {
          float2 v[10];
#pragma unroll
          for (int j = 0; j < 10; ++j)
            if (i0 + j * p.ka < p.P) v[j] = parts[(i0 + j * p.ka) * p.G + g];
#pragma unroll
          for (int j = 0; j < 10; ++j)
            if (i0 + j * p.ka < p.P)
              m.add(i0 + j * p.ka == p.P - 1 ? p.n_last : p.n_full, v[j]);
        }
        if (k == 0) stat[g].x = m.ref;
        if (p.ka == 1)
          stat[g] = mean_rstd(m.finish(p.inv_n), p.inv_n, p.eps);
        else
          sums[k * p.G + g] = make_float2(m.s1, m.s2);
      }
    }
    if (p.ka > 1) {
      __syncthreads();
      const int L = p.lanes_a;  // lanes a group: L * G <= kGnThreads
      const int l = int(threadIdx.x) & (L - 1), g = int(threadIdx.x) >> p.log_lanes_a;
      Merge m{0.0f, 0.0f, 0.0f};
      if (g < p.G) {
        m.ref = stat[g].x;
        for (int j = l; j < p.ka; j += L) {
          m.s1 += sums[j * p.G + g].x;
          m.s2 += sums[j * p.G + g].y;
        }
      }
      for (int o = L >> 1; o > 0; o >>= 1) {
        m.s1 += __shfl_xor_sync(0xffffffffu, m.s1, o);
        m.s2 += __shfl_xor_sync(0xffffffffu, m.s2, o);
      }
      // (the shuffles come after every lane's read of stat[g].x)
      if (l == 0 && g < p.G) stat[g] = mean_rstd(m.finish(p.inv_n), p.inv_n, p.eps);
    }
  }
  __syncthreads();
  for (int c = threadIdx.x; c < p.C; c += kGnThreads) {
    const float2 st = stat[div_small(c, p.magic_cpg)];
    if (c >= kGnThreads) {
      ga = bf16_at(p.gamma, c, 1.0f);
      be = bf16_at(p.beta, c, 0.0f);
    }
    coef[c] = st.x;
    coef[p.C + c] = st.y * ga;
    coef[2 * p.C + c] = be;
  }
  __syncthreads();
  with_act(p.act, [&](auto act) {
    constexpr int ACT = decltype(act)::value;
    Normalize<VEC> nz;
    if (rp < RPa) {
      nz.load(coef, p.C, cv * VEC);
      uint16_t* y = p.Y + base + rp * p.C + cv * VEC;
      int left = cnt;
      while (left >= U) {
        // this batch's rows are in `raw`; the next batch's go out first
        V cur[U];
#pragma unroll
        for (int j = 0; j < U; ++j) cur[j] = raw[j];
        x += U * step;
        left -= U;
        if (left >= U) {
#pragma unroll
          for (int j = 0; j < U; ++j) raw[j] = *reinterpret_cast<const V*>(x + j * step);
        } else {
#pragma unroll
          for (int j = 0; j < U - 1; ++j)
            if (j < left) raw[j] = *reinterpret_cast<const V*>(x + j * step);
        }
#pragma unroll
        for (int j = 0; j < U; ++j) cur[j] = nz.template apply<ACT>(cur[j]);
#pragma unroll
        for (int j = 0; j < U; ++j) *reinterpret_cast<V*>(y + j * step) = cur[j];
        y += U * step;
      }
#pragma unroll
      for (int j = 0; j < U - 1; ++j)
        if (j < left) *reinterpret_cast<V*>(y + j * step) = nz.template apply<ACT>(raw[j]);
    }
    // rows of more than kGnThreads vectors: the other columns
    for (int c2 = nva + int(threadIdx.x); c2 < CV; c2 += kGnThreads) {
      nz.load(coef, p.C, c2 * VEC);
      for (int r = 0; r < rows; ++r) {
        const int64_t off = base + int64_t(r) * p.C + c2 * VEC;
        *reinterpret_cast<V*>(p.Y + off) =
            nz.template apply<ACT>(*reinterpret_cast<const V*>(p.X + off));
      }
    }
  });
}

// The small form: an image's slice of whole groups is one cluster's, which
// holds it in registers.  Each CTA takes a chunk of rows, sends its chunk's
// statistics to every CTA of the cluster, merges all of them in the order of
// the chunks, normalizes and stores.  One launch, X read once.
constexpr int kSmallBytes = 128;  // of X that a thread can hold

template <int VEC>
__global__ void __launch_bounds__(kGnThreads, 1) gn_small_kernel(const GnParams p) {
  extern __shared__ float2 sm[];
  const int M = p.nv * VEC;  // channels of the slice, at most kGnThreads
  float2* part = sm;                                // [VEC][kPartLd]
  float2* sums = sm + VEC * kPartLd;                // [kGnThreads]
  float2* mine = sums + kGnThreads;                 // [gs]
  float2* all = mine + p.gs;                        // [P][gs]
  float* coef = reinterpret_cast<float*>(all + (p.gs << p.log_p));  // [3][M]
  if (p.log_p) asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
  const int chunk = int(blockIdx.x) & (p.P - 1);
  const int unit = int(blockIdx.x) >> p.log_p;
  const int b = unit / p.slices, c0 = (unit - b * p.slices) * M;
  const bool last = chunk == p.P - 1;
  const int rows = last ? p.rows_last : p.rows_p;
  const int nv = p.nv, RP = p.RP;
  const int rp = div_small(int(threadIdx.x), p.magic_nv), cv = int(threadIdx.x) - rp * nv;
  const int q = last ? p.q_last : p.q_full, rem = rows - q * RP;
  const int cnt = rp >= RP ? 0 : rp < rem ? q + 1 : q;
  const int64_t base = (int64_t(b) * p.S + int64_t(chunk) * p.rows_p + rp) * p.C + c0 + cv * VEC;
  const int step = RP * p.C;
  typedef typename Vec<VEC>::T V;
  constexpr int U = kSmallBytes / (2 * VEC);
  V raw[U];
#pragma unroll
  for (int j = 0; j < U; ++j)
    if (j < cnt) raw[j] = *reinterpret_cast<const V*>(p.X + base + j * step);
  float ga = 1.0f, be = 0.0f;
  if (int(threadIdx.x) < M) {
    ga = bf16_at(p.gamma, c0 + int(threadIdx.x), 1.0f);
    be = bf16_at(p.beta, c0 + int(threadIdx.x), 0.0f);
  }
  if (cnt > 0) {
    ThreadStats<VEC> ts;
    ts.start(raw[0]);
#pragma unroll
    for (int j = 1; j < U; ++j)  // (the first value adds nothing around itself)
      if (j < cnt) ts.add(raw[j]);
    ts.finish(cnt, part);
  }
  __syncthreads();
  block_group_stats<VEC>(p, part, sums, min(RP, rows), nv, p.cpg, p.gs,
                         last ? p.inv_n_last : p.inv_n_full, rem, float(q), M, float(rows), 0.0f,
                         p.log_p ? mine : all);
  if (p.log_p) {
    __syncthreads();
    // every CTA of the cluster has started
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
    for (int i = threadIdx.x; i < p.gs << p.log_p; i += kGnThreads) {
      const int g = i >> p.log_p;
      const uint32_t to = mapa_shared(all + chunk * p.gs + g, uint32_t(i & (p.P - 1)));
      st_shared_cluster_u32(to, __float_as_uint(mine[g].x));
      st_shared_cluster_u32(to + 4, __float_as_uint(mine[g].y));
    }
    cluster_sync();
  } else {
    __syncthreads();
  }
  if (int(threadIdx.x) < M) {
    const int c = int(threadIdx.x), g = div_small(c, p.magic_cpg);
    Merge m{all[g].x, 0.0f, 0.0f};
    for (int k = 0; k < p.P; ++k)
      m.add(k == p.P - 1 ? p.n_last : p.n_full, all[k * p.gs + g]);
    const float2 st = mean_rstd(m.finish(p.inv_n), p.inv_n, p.eps);
    coef[c] = st.x;
    coef[M + c] = st.y * ga;
    coef[2 * M + c] = be;
  }
  __syncthreads();
  if (cnt == 0) return;
  with_act(p.act, [&](auto act) {
    constexpr int ACT = decltype(act)::value;
    Normalize<VEC> nz;
    nz.load(coef, M, cv * VEC);
#pragma unroll
    for (int j = 0; j < U; ++j)
      if (j < cnt)
        *reinterpret_cast<V*>(p.Y + base + j * step) = nz.template apply<ACT>(raw[j]);
  });
}

// ---------------------------------------------------------------------- plan
namespace {

int gcd(int a, int b) {
  while (b) {
    const int t = a % b;
    a = b;
    b = t;
  }
  return a;
}

unsigned magic_of(int d) { return d == 1 ? 0u : unsigned(((uint64_t(1) << 32) + d - 1) / d); }

int log2_floor(int v) {
  int l = 0;
  while ((2 << l) <= v) ++l;
  return l;
}

}  // namespace

namespace {

// Per-channel and per-group merging of a CTA's parts (block_group_stats), for
// slices of p->gs groups = p->nv vectors.
void plan_merge(GnParams* p, int vec) {
  const int M = p->nv <= kGnThreads ? p->nv * vec : kGnThreads * vec;
  const int gcpg = M / p->gs;
  p->kk = M >= kGnThreads ? 1 : kGnThreads / M;
  if (p->kk > p->RP) p->kk = p->RP;
  p->magic_m = magic_of(M);
  int lanes = 32;
  while (lanes > 1 && (lanes * p->gs > kGnThreads || lanes >= 2 * gcpg)) lanes >>= 1;
  p->lanes = lanes;
  p->log_lanes = log2_floor(lanes);
}

// The chunks of `rows` rows and what follows from them.
void plan_chunks(GnParams* p, int64_t rows) {
  p->rows_p = int(rows);
  p->P = int((p->S + rows - 1) / rows);
  p->rows_last = int(p->S - (p->P - 1) * rows);
  p->n_full = float(rows) * float(p->cpg);
  p->n_last = float(p->rows_last) * float(p->cpg);
  p->inv_n = float(1.0 / (double(p->S) * p->cpg));
  p->inv_n_full = float(1.0 / (double(rows) * p->cpg));
  p->inv_n_last = float(1.0 / (double(p->rows_last) * p->cpg));
}

// The small form, where a cluster's registers hold an image's slice and all
// clusters run at once, one CTA an SM (clusters of four and eight leave some SMs
// without one).  Modelled time beyond its fixed 4.6 us: what a row a thread
// costs, the cluster's exchange, and slices of less than two sectors.  Fitted to
// sweeps of 1 to 16384 pixels of 64 to 1280 channels in 1 to 140 images (within
// 0.5 us, the choice within 0.3 us of the best).  The two launches take 5 us at
// least and 8 to 9 where this form takes 4.8 to 7.2 (1 x 64 x 1280 8.3 -> 4.8, 4 x
// 1024 x 320 8.0 -> 6.2, 1 x 4096 x 320 8.3 -> 6.9, 30 x 256 x 320 14.8 -> 6.5).
// Narrower vectors lose the gain (3 x 5041 x 182: 8.8 us by two launches, 12.3
// so) and are left to the two launches.
bool gn_small_plan(GnParams* p, int* vec, int sms) {
  if (p->B > sms) return false;
  for (int v : {8, 4}) {
    if (p->C % v != 0) continue;
    const int unit = v / gcd(p->cpg, v);
    double best = 1e30;
    for (int gs = unit; gs <= p->G && gs * p->cpg <= kGnThreads; gs += unit) {
      if (p->G % gs != 0) continue;
      const int RP = kGnThreads / (gs * p->cpg / v);
      // a slice's part of a row: the whole row, at least a sector of 32 bytes, and
      // better two
      const int segment = gs == p->G ? 64 : 2 * gs * p->cpg;
      if (segment < 32) continue;
      for (int lp = 0; lp <= 3; ++lp) {
        if (lp > 0 && p->S < (64 << lp)) break;
        const int64_t rows = (p->S + (1 << lp) - 1) >> lp;
        const int64_t each = (rows + RP - 1) / RP;  // a thread
        const int64_t grid = (p->B * (p->G / gs)) << lp;
        const int64_t at_once = lp == 3 ? sms * 3 / 4 : lp == 2 ? sms * 7 / 8 : sms;
        if (each > kSmallBytes / (2 * v) || grid > at_once || (segment < 64 && each > 4)) continue;
        const double cost = (each <= 3 ? 0.36 * double(each) : 0.42 + 0.22 * double(each)) +
                            (lp > 0 ? 0.5 + 0.05 * lp : 0.0) + (segment < 64 ? 0.8 : 0.0);
        if (cost < best) {
          best = cost;
          p->gs = gs;
          p->log_p = lp;
        }
      }
    }
    if (best < 1e30) {
      *vec = v;
      p->slices = p->G / p->gs;
      plan_chunks(p, (p->S + (1 << p->log_p) - 1) >> p->log_p);
      p->nv = p->gs * p->cpg / v;
      p->RP = kGnThreads / p->nv;
      p->q_full = p->rows_p / p->RP;
      p->q_last = p->rows_last / p->RP;
      p->magic_nv = magic_of(p->nv);
      p->magic_cpg = magic_of(p->cpg);
      plan_merge(p, v);
      return true;
    }
  }
  return false;
}

}  // namespace

// Row chunks and vector width (see GnParams): one CTA an SM over the whole
// batch, two where one leaves more than a tenth of the SMs idle; chunks of less
// than 2^30 elements.
void gn_plan(GnParams* p, int* vec, int sms) {
  const int C = p->C, G = p->G, cpg = C / G;
  p->cpg = cpg;
  p->slices = 0;
  if (gn_small_plan(p, vec, sms)) return;
  // the widest vectors whose slices of whole groups fit a CTA's threads
  for (int v : {8, 4, 2, 1}) {
    if (C % v != 0) continue;
    const int unit = v / gcd(cpg, v);
    if (unit > 1 && int64_t(unit) * cpg / v > kGnThreads) continue;
    *vec = v;
    // as few passes as fit, of equal size up to the vectors' unit
    const int units = G / unit;
    int per = int(int64_t(kGnThreads) * v / (int64_t(unit) * cpg));
    per = per < 1 ? 1 : per > units ? units : per;
    const int passes = (units + per - 1) / per;
    p->gs = (units + passes - 1) / passes * unit;
    break;
  }
  int64_t want = sms / p->B;
  if (want < 1 || double(want * p->B) < 0.9 * sms) want = 2 * int64_t(sms) / p->B;
  const int64_t least = (p->S * C >> 30) + 1;
  want = want > p->S ? p->S : want < least ? least : want;
  const int64_t rows = (p->S + want - 1) / want;
  plan_chunks(p, rows);
  // statistics
  p->nv = p->gs * cpg / *vec;
  p->RP = p->nv <= kGnThreads ? kGnThreads / p->nv : 1;
  p->magic_nv = magic_of(p->nv);
  p->q_full = p->rows_p / p->RP;
  p->q_last = p->rows_last / p->RP;
  plan_merge(p, *vec);
  // normalization
  const int CV = C / *vec;
  p->nva = CV < kGnThreads ? CV : kGnThreads;
  p->RPa = kGnThreads / p->nva;
  p->qa_full = p->rows_p / p->RPa;
  p->qa_last = p->rows_last / p->RPa;
  p->magic_nva = magic_of(p->nva);
  p->magic_g = magic_of(G);
  p->magic_cpg = magic_of(cpg);
  p->ka = G >= kGnThreads ? 1 : kGnThreads / G;
  if (p->ka > p->P) p->ka = p->P;
  int la = 32;
  while (la > 1 && (la * G > kGnThreads || la >= 2 * p->ka)) la >>= 1;
  p->lanes_a = la;
  p->log_lanes_a = log2_floor(la);
}

namespace {

// The shared-memory limit of one kernel, set once on each device.
struct AttrOnce {
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

template <int VEC>
cudaError_t launch_small(const GnParams& p, cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(p.B * p.slices) << p.log_p);
  cfg.blockDim = dim3(kGnThreads);
  cfg.dynamicSmemBytes = sizeof(float2) * (size_t(kPartLd) * VEC + kGnThreads + p.gs +
                                           (size_t(p.gs) << p.log_p)) +
                         sizeof(float) * 3 * size_t(p.nv * VEC);
  cfg.stream = st;
  static AttrOnce once;
  const cudaError_t e = once.set((const void*)gn_small_kernel<VEC>, 80 * 1024);
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute a[1];
  a[0].id = cudaLaunchAttributeClusterDimension;
  a[0].val.clusterDim.x = 1u << p.log_p;
  a[0].val.clusterDim.y = 1;
  a[0].val.clusterDim.z = 1;
  cfg.attrs = a;
  cfg.numAttrs = p.log_p ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, gn_small_kernel<VEC>, p);
}

template <int VEC>
cudaError_t launch_vec(const GnParams& p, cudaStream_t st) {
  if constexpr (VEC >= 4) {
    if (p.slices) return launch_small<VEC>(p, st);
  }
  const int M = p.nv <= kGnThreads ? p.nv * VEC : kGnThreads * VEC;
  const size_t smem_s =
      sizeof(float2) * (size_t(kPartLd) * VEC + size_t(M > kGnThreads ? M : kGnThreads));
  const size_t smem_a = sizeof(float2) * (size_t(p.G) + kGnThreads) + 4 * (3 * size_t(p.C) + 1);
  static AttrOnce as, aa;
  cudaError_t e = as.set((const void*)gn_stats_kernel<VEC>, 80 * 1024);
  if (e == cudaSuccess) e = aa.set((const void*)gn_apply_kernel<VEC>, 176 * 1024);
  if (e != cudaSuccess) return e;
  const unsigned zs = unsigned((p.B + 65534) / 65535);
  const dim3 grid(unsigned(p.P), unsigned(p.B < 65535 ? p.B : 65535), zs);
  gn_stats_kernel<VEC><<<grid, kGnThreads, smem_s, st>>>(p);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(kGnThreads);
  cfg.dynamicSmemBytes = smem_a;
  cfg.stream = st;
  cudaLaunchAttribute a[1];
  a[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  a[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = a;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, gn_apply_kernel<VEC>, p);
}

}  // namespace

cudaError_t launch_group_norm(int vec, const GnParams& p, cudaStream_t st) {
  switch (vec) {
    case 8: return launch_vec<8>(p, st);
    case 4: return launch_vec<4>(p, st);
    case 2: return launch_vec<2>(p, st);
    default: return launch_vec<1>(p, st);
  }
}

}  // namespace hq
