// hq_rows.cu -- the products with an epilogue for a few tokens (T <= 8).
//
//   z[t,n] = sum_k A[t,k] B[n,k],  Y[t,n] = bf16(R + g * act(epilogue(z)))
//
// With so few tokens the product is one pass over B, bound by memory: a tile of
// 128 tokens on the tensor cores would move no more bytes but pays for tensor
// memory, tensor maps and a pipeline before the first byte arrives, and leaves
// most SMs without a tile (4 x 1152 x 6912 in bf16, 16 MB of B: 10.7 us by
// tiles of 128 x 192, 4.8 us by this kernel, B coming from L2; 2 x 256 x 1152
// takes 2.3 us, nearly all of it launch and one trip to memory).  Here B's rows
// go straight from global memory into registers: a warp takes R rows of B and a
// share of K, each lane 16 bytes of each row a step, multiplied by the same 16
// bytes of every token (from L1 after the first row); WK warps share the K of
// the same rows, so that narrow layers still fill the GPU with loads in flight.
//
// Sums: bf16 products are exact in fp32 and summed in fp32 (a lane's steps in
// order, then lanes, then warps: a tree that depends on the sizes alone); int8
// codes are summed exactly by dp4a.  Packed codes are widened to 16 * code as
// they are loaded, and the row scale carries 1/16.
#include <cuda_bf16.h>

#include "hq_act.cuh"
#include "hq_device.cuh"
#include "hq_kernels.h"

namespace hq {

namespace {

constexpr int kRowsBF16 = 0, kRowsI8 = 1, kRowsI4 = 2;  // operand kinds (I4: packed A)
constexpr int kRowsThreads = 128;

// The sum of the element products of 16 bytes of a row of B and of a token.
template <int KIND>
struct Acc;
template <>
struct Acc<kRowsBF16> {
  typedef float T;
  // two partial sums, of the even and of the odd elements, in one pair
  f2 v = {0.0f, 0.0f};
  __device__ __forceinline__ void add(const uint4& b, const uint4& a) {
    const uint32_t x[4] = {a.x, a.y, a.z, a.w}, w[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) v = fma2(unpack_bf16x2(w[i]), unpack_bf16x2(x[i]), v);
  }
  __device__ __forceinline__ float sum() const { return v.x + v.y; }
};
template <>
struct Acc<kRowsI8> {
  typedef int T;
  int v = 0;
  __device__ __forceinline__ void add(const uint4& b, const uint4& a) {
    v = __dp4a(int(b.x), int(a.x), v);
    v = __dp4a(int(b.y), int(a.y), v);
    v = __dp4a(int(b.z), int(a.z), v);
    v = __dp4a(int(b.w), int(a.w), v);
  }
  __device__ __forceinline__ int sum() const { return v; }
};
template <>
struct Acc<kRowsI4> : Acc<kRowsI8> {};

// 16 elements-bytes of a token at byte offset `k` of a row of B.
template <int KIND>
__device__ __forceinline__ uint4 load_a(const uint8_t* row, int k) {
  if constexpr (KIND == kRowsI4) {
    // eight packed bytes -> 16 int8 values 16 * code, in element order
    const uint2 p = *reinterpret_cast<const uint2*>(row + k / 2);
    uint4 v;
    const uint32_t e0 = (p.x << 4) & 0xF0F0F0F0u, o0 = p.x & 0xF0F0F0F0u;
    const uint32_t e1 = (p.y << 4) & 0xF0F0F0F0u, o1 = p.y & 0xF0F0F0F0u;
    v.x = __byte_perm(e0, o0, 0x5140);
    v.y = __byte_perm(e0, o0, 0x7362);
    v.z = __byte_perm(e1, o1, 0x5140);
    v.w = __byte_perm(e1, o1, 0x7362);
    return v;
  } else {
    return *reinterpret_cast<const uint4*>(row + k);
  }
}

// Sums v[0 .. NV) over the warp's lanes; lane l returns the total of value
// l / (32 / NV).  Each step halves the values a lane holds: NV - 1 + log2(32/NV)
// exchanges instead of 5 NV.
template <int NV, class T>
__device__ __forceinline__ T warp_reduce(T (&v)[NV], int lane) {
  int o = 16;
#pragma unroll
  for (int n = NV / 2; n >= 1; n /= 2, o /= 2) {
    const bool up = lane & o;
#pragma unroll
    for (int i = 0; i < n; ++i) {
      const T mine = up ? v[i + n] : v[i];
      const T give = up ? v[i] : v[i + n];
      v[i] = mine + __shfl_xor_sync(0xffffffffu, give, o);
    }
  }
  T s = v[0];
#pragma unroll
  for (; o >= 1; o /= 2) s += __shfl_xor_sync(0xffffffffu, s, o);
  return s;
}

}  // namespace

// A CTA: wr groups of R rows (p.wr), each shared by wk = 4 / wr warps over K.
// TT: tokens, T <= TT.
template <int KIND, int TT, int R>
__global__ void __launch_bounds__(kRowsThreads) rows_kernel(const RowsParams p) {
  typedef typename Acc<KIND>::T S;
  constexpr int NV = R * TT;
  __shared__ S part[kRowsThreads / 32][NV];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int wk = (kRowsThreads / 32) >> p.log_wr;
  const int group = warp >> (2 - p.log_wr);  // warps of a group are neighbours
  const int kw = warp & (wk - 1);
  const int n0 = (int(blockIdx.x) * (1 << p.log_wr) + group) * R;
  Acc<KIND> acc[R][TT];
  {
    const uint8_t* brow[R];
#pragma unroll
    for (int r = 0; r < R; ++r)
      brow[r] = p.B + int64_t(n0 + r < p.N ? n0 + r : p.N - 1) * p.row_bytes;
    const uint8_t* arow[TT];
#pragma unroll
    for (int t = 0; t < TT; ++t) arow[t] = p.A + int64_t(t < p.T ? t : p.T - 1) * p.a_row_bytes;
    const int step = wk * 512;
    int k = kw * 512 + lane * 16;
    // U steps at a time: U R loads of B in flight a lane
    constexpr int U = TT <= 2 ? 4 : TT == 4 ? 2 : 1;
    for (; k + (U - 1) * step < p.row_bytes; k += U * step) {
      uint4 b[U][R], a[TT];
#pragma unroll
      for (int j = 0; j < U; ++j)
#pragma unroll
        for (int r = 0; r < R; ++r)
          b[j][r] = __ldg(reinterpret_cast<const uint4*>(brow[r] + k + j * step));
#pragma unroll
      for (int j = 0; j < U; ++j) {
#pragma unroll
        for (int t = 0; t < TT; ++t) a[t] = load_a<KIND>(arow[t], k + j * step);
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
          for (int t = 0; t < TT; ++t) acc[r][t].add(b[j][r], a[t]);
      }
    }
    if constexpr (U > 1) {  // the rest, at most U - 1 steps, loaded at once
      uint4 b[U - 1][R], a[TT];
#pragma unroll
      for (int j = 0; j < U - 1; ++j)
#pragma unroll
        for (int r = 0; r < R; ++r)
          b[j][r] = k + j * step < p.row_bytes
                        ? __ldg(reinterpret_cast<const uint4*>(brow[r] + k + j * step))
                        : make_uint4(0, 0, 0, 0);
#pragma unroll
      for (int j = 0; j < U - 1; ++j) {
        if (k + j * step < p.row_bytes) {
#pragma unroll
          for (int t = 0; t < TT; ++t) a[t] = load_a<KIND>(arow[t], k + j * step);
#pragma unroll
          for (int r = 0; r < R; ++r)
#pragma unroll
            for (int t = 0; t < TT; ++t) acc[r][t].add(b[j][r], a[t]);
        }
      }
    }
  }
  S v[NV];
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int t = 0; t < TT; ++t) v[t * R + r] = acc[r][t].sum();
  S total = warp_reduce<NV>(v, lane);
  const int idx = lane / (32 / NV);
  if (wk > 1) {
    if (lane % (32 / NV) == 0) part[warp][idx] = total;
    __syncthreads();
    if (kw != 0) return;
    for (int w = 1; w < wk; ++w) total += part[warp + w][idx];
  }
  const int t = idx / R, n = n0 + idx % R;
  if (lane % (32 / NV) != 0 || t >= p.T || n >= p.N) return;
  float z;
  if constexpr (KIND == kRowsBF16) {
    z = total + (p.bias16 ? __uint_as_float(uint32_t(p.bias16[n]) << 16) : 0.0f);
  } else {
    const float sx = (p.a_scale_per_row ? p.a_scale[t] : p.a_scale[0]) * p.acc_unit;
    float c = p.bias ? p.bias[n] : 0.0f;
    if (p.a_mean) c = fmaf(p.a_mean[t], p.colsum[n], c);
    z = fmaf(__int2float_rn(total), sx * p.w_scale[n], c);
  }
  f2 zz[1] = {pk(z, 0.0f)};
  act_chunk(p.act, zz);
  z = zz[0].x;
  const int64_t off = int64_t(t) * p.N + n;
  if (p.gate)
    z *= __uint_as_float(uint32_t(p.gate[(p.gate_rows == 1 ? t : t / p.gate_rows) * p.N + n]) << 16);
  if (p.residual) z += __uint_as_float(uint32_t(p.residual[off]) << 16);
  p.Y[off] = uint16_t(pack_bf16x2(z, 0.0f) & 0xFFFFu);
}

namespace {

// Rows of B a warp: two for one or two tokens; four for more, which halves the
// tokens' reads from L1.
constexpr int rows_per_warp(int T) { return T > 2 ? 4 : 2; }

template <int KIND, int TT, int R>
cudaError_t launch_one(const RowsParams& p, cudaStream_t st) {
  const int rows = R << p.log_wr;
  rows_kernel<KIND, TT, R><<<(p.N + rows - 1) / rows, kRowsThreads, 0, st>>>(p);
  return cudaGetLastError();
}

template <int KIND>
cudaError_t launch_tt(const RowsParams& p, cudaStream_t st) {
  if (p.T == 1) return launch_one<KIND, 1, rows_per_warp(1)>(p, st);
  if (p.T == 2) return launch_one<KIND, 2, rows_per_warp(2)>(p, st);
  if (p.T <= 4) return launch_one<KIND, 4, rows_per_warp(4)>(p, st);
  return launch_one<KIND, 8, rows_per_warp(8)>(p, st);
}

}  // namespace

int rows_warps(int T, int N, int64_t row_bytes, int sms) {
  // K is shared between two or four warps while there are fewer than eight warps
  // an SM, and up to sixteen where it leaves each the four steps it keeps in
  // flight.  (Measured over 1152..16384 outputs and 256..4608 inputs; within 10 %
  // of the best of the six choices of this and of the rows a warp.)
  const int r = rows_per_warp(T);
  int log_wk = 0;
  while (log_wk < 2 && (int64_t(2) << log_wk) * 512 <= row_bytes) {
    const int64_t warps = (int64_t(N) / r) << log_wk;
    if (warps >= 16 * int64_t(sms) ||
        (warps >= 8 * int64_t(sms) && (int64_t(2) << log_wk) * 2048 > row_bytes))
      break;
    ++log_wk;
  }
  return 1 << log_wk;
}

cudaError_t launch_rows(int kind, RowsParams p, int wk, cudaStream_t st) {
  p.log_wr = wk == 1 ? 2 : wk == 2 ? 1 : 0;
  switch (kind) {
    case kRowsBF16: return launch_tt<kRowsBF16>(p, st);
    case kRowsI8: return launch_tt<kRowsI8>(p, st);
    default: return launch_tt<kRowsI4>(p, st);
  }
}

}  // namespace hq
