// hq_gemm_tile.cuh -- tiled GEMM with a fused epilogue on 5th-generation tensor
// cores (tcgen05, accumulators in tensor memory): the device code behind the
// integer GEMM (hq_gemm.cu) and the products with an activation, a gate and a
// residual in their epilogue (hq_gemm_ep.cu).
//
// The integer GEMM (kind::i8, int32 accumulators):
//
//   acc[t,n] = sum_k A[t,k] * B[n,k]                 (HaTQ Sec. IV-B Eq. (14))
//   Y[t,n]   = bf16( s_x[t] * s_w[n] * acc[t,n]      (accumulator scale, HaTQ Eq. (18))
//                    + b[n] + mu_t * colsum[n] )      (b~ = b + mu W~, HadaNorm Eq. (1))
//
// A = activation codes [T,K] int8 (or two 4-bit codes per byte, see PK
// below), B = weight codes [N,K] int8, both K-major.
// Two kernels share one warp layout (320 threads, one CTA per SM; the packed
// form adds warps 10..13):
//   warp 0      one thread issues TMA tensor loads (128-byte swizzle) of the
//               A and B K-slices into a ring of shared-memory stages, and per
//               output tile bulk copies of the tile's columns of s_w, colsum
//               and bias into a two-slot parameter ring;
//   warp 1      allocates tensor memory; one thread issues tcgen05.mma and
//               commits each stage back to the producer and each finished
//               accumulator to the epilogue;
//   warps 2..9  the epilogue: two warps per 32-lane quarter of tensor memory,
//               each taking half of the tile's columns.  A warp reads its
//               columns of the accumulator (tcgen05.ld, up to three 32-column
//               chunks per wait) and hands the accumulator back to the MMA
//               issuer as soon as the last read has landed; then per chunk it
//               applies the epilogue in fp32 (row scale and mean from
//               registers, prefetched one tile ahead; column parameters from
//               the ring), writes bf16 to a 64-byte swizzled shared buffer and
//               lets a TMA tensor store write the 32 x 32 box to Y (clipped at
//               the tensor's edges).
//
// gemm_body<KIND, BN, LOGO, PK, EP>: one CTA per 128 x BN output tile (BN
//   64..256).
//   LOGO > 0 selects the weight-only Hadamard epilogue (HaTQ Sec. IV-B
//   Eq. (17)): Y = (s_x s_w acc) H_out + b, the fast Walsh-Hadamard transform
//   over each block of 2^LOGO output columns done in registers after the
//   dequantization (no mean term: that form has no centering).
//   PK: A holds two 4-bit codes per byte.  TMA loads each stage's 128 x
//   64-byte packed tile (64-byte swizzle) next to B; four more warps (warps
//   10..13, one per 32-lane quarter of tensor memory) each read their rows'
//   packed bytes, widen them to int8 (each nibble moved to the high half of
//   its byte: 16 * code, sign included) and store them with tcgen05.st into
//   tensor memory, where the MMA takes its A operand; a third barrier hands
//   the stage to the MMA issuer.  The accumulator is then 16 times the code
//   products' sum, exactly; the epilogue's row scale carries the factor
//   1/16.  No tensor-core kind multiplies 4-bit integers on sm_100a; with A
//   in tensor memory the widened tile never passes through shared memory,
//   whose traffic (tensor loads in, MMA operand reads out) bounds the main
//   loop, so the packed stage costs less shared-memory traffic than an int8
//   one.  A's stages sit in tensor memory after the two accumulators, so
//   packed tiles are at most 192 columns wide.
// gemm_pair_body<KIND, BN, EP>: a cluster of two CTAs per 256 x BN output tile with
//   the CTA-pair MMA (cta_group::2, M = 256): each CTA loads 128 rows of A and
//   BN / 2 rows of B into its own shared memory, so one SM moves half the B
//   bytes per MMA that the single-CTA kernel moves.  Both CTAs' copies
//   complete on the even CTA's stage barrier, whose producer expects the
//   bytes of both; the even CTA issues the MMAs and commits to both CTAs.
// KIND kBF16 multiplies bf16 operands (kind::f16, fp32 accumulators) with the
//   same byte geometry: a stage is 128 bytes of K (64 elements), an MMA step
//   32 bytes (16 elements), and p.K counts bytes.
// EP adds to the epilogue  Y = bf16(R + g * act(z))  (see epi_tile_ep): z is
//   the value that the plain epilogue would round, act an elementwise
//   activation in fp32, g a row of gate values shared by gate_rows rows of Y,
//   R the residual.  The activation makes the epilogue as long as a short main
//   loop, so these kernels run up to sixteen epilogue warps (64 columns each)
//   instead of eight.
// Two accumulators in tensor memory let the epilogue of one tile overlap the
// main loop of the next.  Every wait is bounded; a timeout records
// HQ_ERR_TIMEOUT in the device error word, and the CTA waits for every copy it
// started (or, in the pair kernel, the even CTA for the pair's copies) before
// it exits.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>

#include <type_traits>

#include "hq_act.cuh"
#include "hq_device.cuh"
#include "hq_kernels.h"

namespace hq {

namespace {

constexpr int BM = 128;
constexpr int BK = 128;  // K bytes per stage: one 128-byte swizzle row
constexpr int kEpiWarps = 8;
constexpr int kGemmThreads = 64 + 32 * kEpiWarps;
constexpr int kConvWarps = 4;  // packed-A converters of the single-CTA kernel (one per lane quarter)
constexpr int kSmemLimit = 227 * 1024;
constexpr int kStageBox = 2048;           // one 32 x 32 bf16 output box
constexpr float kAccMagic = 12582912.0f;  // 1.5 * 2^23
constexpr int kAccMagicBits = 0x4B400000;

// instruction descriptor: D s32 (bits 4-5 = 2), A and B signed int8 (bits
// 7-9 = 1, 10-12 = 1), both K-major, N >> 3 at bits 17-22, M >> 4 at 24-28.
constexpr uint32_t i8_idesc(int m, int n) {
  return (2u << 4) | (1u << 7) | (1u << 10) | (uint32_t(n >> 3) << 17) | (uint32_t(m >> 4) << 24);
}
// the same with D fp32 (bits 4-5 = 1) and bf16 operands (format 1)
constexpr uint32_t bf16_idesc(int m, int n) {
  return (1u << 4) | (1u << 7) | (1u << 10) | (uint32_t(n >> 3) << 17) | (uint32_t(m >> 4) << 24);
}

// Operand kinds.
constexpr int kI8 = 0;    // int8 codes -> int32 accumulators
constexpr int kBF16 = 1;  // bf16 -> fp32 accumulators

template <int KIND>
__device__ __forceinline__ void mma_kind(uint32_t d_tmem, uint64_t a, uint64_t b, uint32_t idesc,
                                         uint32_t accumulate) {
  if constexpr (KIND == kBF16)
    mma_bf16(d_tmem, a, b, idesc, accumulate);
  else
    mma_i8(d_tmem, a, b, idesc, accumulate);
}
template <int KIND>
__device__ __forceinline__ void mma_kind_pair(uint32_t d_tmem, uint64_t a, uint64_t b,
                                              uint32_t idesc, uint32_t accumulate) {
  if constexpr (KIND == kBF16)
    mma_bf16_pair(d_tmem, a, b, idesc, accumulate);
  else
    mma_i8_pair(d_tmem, a, b, idesc, accumulate);
}

template <bool EP>
using GemmArgs = std::conditional_t<EP, GemmEpParams, GemmParams>;

constexpr int tmem_cols_for(int cols) {
  return cols <= 32 ? 32 : cols <= 64 ? 64 : cols <= 128 ? 128 : cols <= 256 ? 256 : 512;
}

// Shared-memory matrix descriptor for a K-major operand tile written by TMA
// with 128-byte swizzling: rows of 128 bytes, 8-row (1024-byte) swizzle atoms
// stacked along M/N (stride byte offset 1024), leading byte offset unused (1),
// descriptor version 1, layout type 2 (128-byte swizzle).
__device__ __forceinline__ uint64_t sw128_kmajor_desc(uint32_t saddr) {
  uint64_t d = 0;
  d |= uint64_t((saddr & 0x3FFFFu) >> 4);
  d |= uint64_t(1) << 16;
  d |= uint64_t(1024 >> 4) << 32;
  d |= uint64_t(1) << 46;
  d |= uint64_t(2) << 61;
  return d;
}

// Output tile `tile` -> (M tile, N tile) in groups of p.group_m M tiles: the
// tiles of a group run N tile by N tile over the group's M tiles, so the CTAs
// working at one time share a few M tiles of A and a few N tiles of B, which
// stay in L2 while the output streams past (plain M-fastest order sweeps all
// of A every round of tiles, and the output evicts it).
__device__ __forceinline__ int tile_m(const GemmParams& p, int tile) {
  const int gsize = p.group_m * p.num_n_tiles;
  const int first = (tile / gsize) * p.group_m;
  const int gm = min(p.num_m_tiles - first, p.group_m);
  return first + (tile % gsize) % gm;
}
__device__ __forceinline__ int tile_n(const GemmParams& p, int tile) {
  const int gsize = p.group_m * p.num_n_tiles;
  const int first = (tile / gsize) * p.group_m;
  const int gm = min(p.num_m_tiles - first, p.group_m);
  return (tile % gsize) / gm;
}

// ------------------------------------------------------- parameter ring
// Slot a holds the columns [n0, n0 + W) of one output tile: s_w at [0, W),
// colsum at [W, 2W), bias at [2W, 3W) (fp32).  An absent vector, and every
// column past N, reads zero or a finite stale value: the ring is zeroed at
// kernel start and absent vectors are never copied.
template <int W>
__device__ __forceinline__ void param_ring_zero(float* ring, int tid, int nthreads) {
  for (int i = tid; i < 2 * 3 * W; i += nthreads) ring[i] = 0.0f;
}

// Producer side: copies the tile's columns [n0, min(n0 + W, N)) into `slot`,
// completion counted on `bar`.
template <int W>
__device__ __forceinline__ void param_ring_load(const GemmParams& p, float* slot, int n0,
                                                uint64_t* bar) {
  const int cols = p.N - n0 < W ? p.N - n0 : W;
  const uint32_t nb = uint32_t(cols) * 4u;  // N % 16 == 0: a multiple of 64 bytes
  const bool cs = p.a_mean != nullptr && p.colsum != nullptr;
  const bool bi = p.bias != nullptr;
  mbar_arrive_expect_tx(bar, nb * (1u + (cs ? 1u : 0u) + (bi ? 1u : 0u)));
  bulk_load(slot, p.w_scale + n0, nb, bar);
  if (cs) bulk_load(slot + W, p.colsum + n0, nb, bar);
  if (bi) bulk_load(slot + 2 * W, p.bias + n0, nb, bar);
}

// The same for bf16 operands: the tile's columns of the bf16 bias at the
// start of the slot (N % 8 == 0: a multiple of 16 bytes).
template <int W>
__device__ __forceinline__ void param_ring_load16(const GemmEpParams& p, float* slot, int n0,
                                                  uint64_t* bar) {
  const int cols = p.N - n0 < W ? p.N - n0 : W;
  const uint32_t nb = p.bias16 != nullptr ? uint32_t(cols) * 2u : 0u;
  mbar_arrive_expect_tx(bar, nb);
  if (nb) bulk_load(slot, p.bias16 + n0, nb, bar);
}

// ------------------------------------------------------- packed A operand
// One word of eight 4-bit two's-complement codes (element 2j in the low
// nibble of byte j) -> two words of eight int8 values 16 * code, in element
// order: each nibble moved to the high half of its own byte is already the
// sign-extended code times 16, so no sign extension is needed.
__device__ __forceinline__ void widen_i4x8(uint32_t v, uint32_t& lo, uint32_t& hi) {
  const uint32_t ev = (v << 4) & 0xF0F0F0F0u;  // elements 0, 2, 4, 6
  const uint32_t od = v & 0xF0F0F0F0u;         // elements 1, 3, 5, 7
  lo = __byte_perm(ev, od, 0x5140);
  hi = __byte_perm(ev, od, 0x7362);
}

// ------------------------------------------------------------- epilogue
// Per-warp state of the epilogue for one output tile.
struct EpiTile {
  int row0;      // first output row of this warp's 32 rows
  int col_base;  // first output column of this warp's columns
  int64_t row;   // this thread's output row
  bool row_ok;   // row < T
  float sx, mt;  // this row's activation scale and mean
};

// This thread's row scale and mean (zero past T).
__device__ __forceinline__ void load_row_params(const GemmParams& p, int64_t row, float& sx,
                                                float& mt) {
  sx = 0.0f;
  mt = 0.0f;
  if (row < p.T) {
    // packed A enters the MMA as 16 * code, so the accumulator is 16 times
    // the code products' sum; times acc_unit = 1/16 (exact) undoes it
    sx = (p.a_scale_per_row ? p.a_scale[row] : p.a_scale[0]) * p.acc_unit;
    mt = p.a_mean ? p.a_mean[row] : 0.0f;
  }
}

// Raw accumulators of chunk c to acc_debug (bit-exact checks), when asked for.
__device__ __forceinline__ void epi_acc_debug(const GemmParams& p, const uint32_t (&r)[32], int c,
                                              const EpiTile& e) {
  if (p.acc_debug && e.row_ok) {
    const int col0 = e.col_base + c * 32;
    int32_t* arow = p.acc_debug + e.row * p.N;
#pragma unroll
    for (int g = 0; g < 8; ++g) {
      if (col0 + 4 * g < p.N) {
        const int sh = p.acc_shift;  // exact: a packed A's accumulator is a multiple of 16
        *reinterpret_cast<int4*>(arow + col0 + 4 * g) =
            make_int4(int(r[4 * g]) >> sh, int(r[4 * g + 1]) >> sh, int(r[4 * g + 2]) >> sh,
                      int(r[4 * g + 3]) >> sh);
      }
    }
  }
}

// One 32-column chunk c of the warp's columns: accumulators r (this thread's
// row) -> fp32 values z.  prm points at the warp's first column in a parameter
// slot of width W.
template <int W>
__device__ __forceinline__ void epi_z(const GemmParams& p, const uint32_t (&r)[32], int c,
                                         const EpiTile& e, const float* prm,
                                         f2 (&z)[16]) {
  const float* pw = prm + c * 32;
  const f2 sx2 = pk(e.sx, e.sx), mt2 = pk(e.mt, e.mt);
#pragma unroll
  for (int g = 0; g < 8; ++g) {
    const float4 sw = *reinterpret_cast<const float4*>(pw + 4 * g);
    const float4 cs = *reinterpret_cast<const float4*>(pw + W + 4 * g);
    const float4 bb = *reinterpret_cast<const float4*>(pw + 2 * W + 4 * g);
    f2 a01, a23;
    if (p.small_acc) {
      // |acc| < 2^22: acc + 1.5*2^23 is exact in fp32, so subtracting the
      // magic constant recovers float(acc) without the conversion unit
      const f2 mg = pk(kAccMagic, kAccMagic);
      a01 = sub2(pk(__int_as_float(int(r[4 * g + 0]) + kAccMagicBits),
                    __int_as_float(int(r[4 * g + 1]) + kAccMagicBits)), mg);
      a23 = sub2(pk(__int_as_float(int(r[4 * g + 2]) + kAccMagicBits),
                    __int_as_float(int(r[4 * g + 3]) + kAccMagicBits)), mg);
    } else {
      a01 = pk(__int2float_rn(int(r[4 * g + 0])), __int2float_rn(int(r[4 * g + 1])));
      a23 = pk(__int2float_rn(int(r[4 * g + 2])), __int2float_rn(int(r[4 * g + 3])));
    }
    // y = acc * (s_x * s_w) + (b + m * colsum)
    z[2 * g] = fma2(a01, mul2(sx2, pk(sw.x, sw.y)), fma2(mt2, pk(cs.x, cs.y), pk(bb.x, bb.y)));
    z[2 * g + 1] = fma2(a23, mul2(sx2, pk(sw.z, sw.w)), fma2(mt2, pk(cs.z, cs.w), pk(bb.z, bb.w)));
  }
  epi_acc_debug(p, r, c, e);
}

// The same for bf16 operands: z = acc + b.  prm: the warp's columns of the
// bf16 bias.
__device__ __forceinline__ void epi_z_bf16(const uint32_t (&r)[32], int c, const uint16_t* prm,
                                           f2 (&z)[16]) {
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const uint4 b = *reinterpret_cast<const uint4*>(prm + c * 32 + 8 * q);
    const uint32_t w[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
    for (int i = 0; i < 4; ++i)
      z[4 * q + i] = add2(pk(__uint_as_float(r[8 * q + 2 * i]), __uint_as_float(r[8 * q + 2 * i + 1])),
                          unpack_bf16x2(w[i]));
  }
}

__device__ __forceinline__ void pack_chunk(const f2 (&z)[16], uint32_t (&packed)[16]) {
#pragma unroll
  for (int i = 0; i < 16; ++i) packed[i] = pack_bf16x2(z[i].x, z[i].y);
}

// Weight-only Hadamard form, step 1 for chunk c: z = acc * (s_x * s_w) in the
// output Hadamard basis (no mean term: the form has no centering).
template <int W>
__device__ __forceinline__ void epi_dequant(const GemmParams& p, const uint32_t (&r)[32], int c,
                                            const EpiTile& e, const float* prm, f2 (&z)[16]) {
  const float* pw = prm + c * 32;
  const f2 sx2 = pk(e.sx, e.sx);
#pragma unroll
  for (int g = 0; g < 8; ++g) {
    const float4 sw = *reinterpret_cast<const float4*>(pw + 4 * g);
    f2 a01, a23;
    if (p.small_acc) {
      const f2 mg = pk(kAccMagic, kAccMagic);
      a01 = sub2(pk(__int_as_float(int(r[4 * g + 0]) + kAccMagicBits),
                    __int_as_float(int(r[4 * g + 1]) + kAccMagicBits)), mg);
      a23 = sub2(pk(__int_as_float(int(r[4 * g + 2]) + kAccMagicBits),
                    __int_as_float(int(r[4 * g + 3]) + kAccMagicBits)), mg);
    } else {
      a01 = pk(__int2float_rn(int(r[4 * g + 0])), __int2float_rn(int(r[4 * g + 1])));
      a23 = pk(__int2float_rn(int(r[4 * g + 2])), __int2float_rn(int(r[4 * g + 3])));
    }
    z[2 * g] = mul2(a01, mul2(sx2, pk(sw.x, sw.y)));
    z[2 * g + 1] = mul2(a23, mul2(sx2, pk(sw.z, sw.w)));
  }
  epi_acc_debug(p, r, c, e);
}

// Unnormalized fast Walsh-Hadamard transform over blocks of 2^LOGB (<= 32)
// consecutive columns of a chunk held as 16 column pairs: index bit 0 inside
// each pair, bits 1 .. LOGB-1 between pairs.
template <int LOGB>
__device__ __forceinline__ void fwht_chunk(f2 (&z)[16]) {
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const float a = z[i].x, b = z[i].y;
    z[i] = pk(__fadd_rn(a, b), __fsub_rn(a, b));
  }
#pragma unroll
  for (int bit = 1; bit < LOGB; ++bit) {
    const int hh = 1 << (bit - 1);
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      if ((i & hh) == 0) {
        const f2 x = z[i], y = z[i + hh];
        z[i] = add2(x, y);
        z[i + hh] = sub2(x, y);
      }
    }
  }
}

// Weight-only Hadamard form, last step for chunk c: z / sqrt(m) + b in the
// original output basis, in place.
template <int W>
__device__ __forceinline__ void epi_finish(const GemmParams& p, f2 (&z)[16], int c,
                                           const float* prm) {
  const float* pw = prm + c * 32;
  const f2 inv2 = pk(p.inv_sqrt_out, p.inv_sqrt_out);
#pragma unroll
  for (int g = 0; g < 8; ++g) {
    const float4 bb = *reinterpret_cast<const float4*>(pw + 2 * W + 4 * g);
    z[2 * g] = fma2(z[2 * g], inv2, pk(bb.x, bb.y));
    z[2 * g + 1] = fma2(z[2 * g + 1], inv2, pk(bb.z, bb.w));
  }
}

// Chunk c's bf16 values into staging box `buf` (64-byte swizzled rows), then
// one thread stores the 32 x 32 box to Y (clipped at the tensor's edges) as
// its own bulk group.
__device__ __forceinline__ void epi_store_chunk(const GemmParams& p, const CUtensorMap* tmY,
                                                const uint32_t (&packed)[16], int col0, int row0,
                                                uint8_t* buf, int lane) {
  const int swz = (lane >> 1) & 3;  // 64-byte swizzle of this thread's row
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    *reinterpret_cast<uint4*>(buf + lane * 64 + ((q ^ swz) << 4)) =
        make_uint4(packed[4 * q], packed[4 * q + 1], packed[4 * q + 2], packed[4 * q + 3]);
  }
  fence_proxy_async_smem();
  __syncwarp();
  if (lane == 0 && col0 < p.N && row0 < p.T) {
    tma_store_2d(tmY, buf, col0, row0);
    bulk_commit_group();
  }
}

// The warp's HC columns (HC / 32 chunks) of one accumulator at tensor-memory
// address t_addr (lane quarter already encoded), through NBOX staging boxes
// of kStageBox bytes:
//   - the chunks are read from tensor memory in groups of up to three per
//     wait (96 accumulator registers); right after the last group's wait
//     `release_acc` hands the accumulator back to the MMA issuer, so the
//     next main loop into it can start while this tile is still being stored;
//   - per chunk: the epilogue arithmetic, then a wait until the store that
//     last used the chunk's box has read it, then the box and its TMA store;
//   - `release_params` frees the parameter slot after the last chunk's
//     arithmetic.
// LOGO > 0 selects the weight-only Hadamard epilogue with output blocks of
// 2^LOGO columns (4, 5 or 6): dequantize, a fast Walsh-Hadamard transform
// over each block (inside a chunk, and for 64-column blocks one more stage
// between the two chunks of a group), then 1/sqrt(m) and the bias.
template <int HC, int W, int NBOX, int LOGO, int GMAX, class RelAcc, class RelPrm>
__device__ __forceinline__ void epi_tile(const GemmParams& p, const CUtensorMap* tmY,
                                         uint32_t t_addr, const EpiTile& e, const float* prm,
                                         uint8_t* stg, int lane, RelAcc release_acc,
                                         RelPrm release_params) {
  constexpr int NCH = HC / 32;
  constexpr int G0 = NCH <= 3 ? NCH : 2;
  constexpr int G = G0 <= GMAX ? G0 : (NCH % 2 == 0 && GMAX >= 2 ? 2 : 1);
  static_assert(NCH % G == 0, "whole groups of chunks");
  static_assert(LOGO == 0 || (LOGO >= 4 && LOGO <= 5) || (LOGO == 6 && G % 2 == 0),
                "output blocks of 16 or 32 columns, or 64 over chunk pairs");
#pragma unroll
  for (int c0 = 0; c0 < NCH; c0 += G) {
    uint32_t r[G][32];
#pragma unroll
    for (int c = 0; c < G; ++c) tmem_ld_32x32b_x32(t_addr + uint32_t((c0 + c) * 32), r[c]);
    tmem_wait_ld();
    if (c0 + G == NCH) release_acc();
    if constexpr (LOGO == 0) {
#pragma unroll
      for (int c = 0; c < G; ++c) {
        const int ch = c0 + c;
        f2 z[16];
        uint32_t packed[16];
        epi_z<W>(p, r[c], ch, e, prm, z);
        pack_chunk(z, packed);
        if (ch == NCH - 1) release_params();
        if (lane == 0) bulk_wait_group_read<NBOX - 1>();
        __syncwarp();
        epi_store_chunk(p, tmY, packed, e.col_base + ch * 32, e.row0,
                        stg + (ch % NBOX) * kStageBox, lane);
      }
    } else {
      f2 z[G][16];
#pragma unroll
      for (int c = 0; c < G; ++c) {
        epi_dequant<W>(p, r[c], c0 + c, e, prm, z[c]);
        fwht_chunk<(LOGO < 5 ? LOGO : 5)>(z[c]);
      }
      if constexpr (LOGO == 6) {
        // index bit 5: between the two 32-column chunks of each pair
#pragma unroll
        for (int c = 0; c < G; c += 2) {
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const f2 x = z[c][i], y = z[c + 1][i];
            z[c][i] = add2(x, y);
            z[c + 1][i] = sub2(x, y);
          }
        }
      }
#pragma unroll
      for (int c = 0; c < G; ++c) {
        const int ch = c0 + c;
        uint32_t packed[16];
        epi_finish<W>(p, z[c], ch, prm);
        pack_chunk(z[c], packed);
        if (ch == NCH - 1) release_params();
        if (lane == 0) bulk_wait_group_read<NBOX - 1>();
        __syncwarp();
        epi_store_chunk(p, tmY, packed, e.col_base + ch * 32, e.row0,
                        stg + (ch % NBOX) * kStageBox, lane);
      }
    }
  }
}

// ------------------------------------- epilogue with activation and residual
// Two layouts, by the tile (kWide): shared memory holds either more stages or
// more epilogue.
//   wide (tiles of up to 192 columns): a warp owns 32 rows x 64 columns and one
//     staging box of that shape (4 KB, 128-byte rows, 128-byte swizzle).  R's
//     box arrives in it by TMA, is added to in place, and leaves by TMA as Y's;
//     the next tile's box of R is fetched as soon as the store has read the
//     box, and so travels during the next main loop.  For short main loops,
//     where the epilogue's arithmetic is the longer part.
//   lean (256 columns and the CTA pair): eight warps of 128 columns with one
//     32 x 32 box each, so that the operands keep four stages of 48 KB (six of
//     32 KB in the pair); R comes from global memory into registers one chunk
//     ahead.  For long main loops: 16384 x 4096 x 8192 in bf16 takes 742-800 us
//     so in short runs (870 where the power cap holds the clock down), 843-869 us
//     with sixteen warps, 64 KB of boxes and four stages.  In between, 16384 x 1152
//     x 4608 in bf16: 134 us by the lean pair, 148 by the wide pair of 192 columns.
// (Stores from registers, 32 bytes a thread and row, were tried: the 32
// single-sector accesses of a warp instruction made the epilogue of a 128 x 256
// tile 11000 cycles instead of 7000.  Sixteen warps of 32 columns on tiles of
// 128 columns have 96 registers a thread and spill: 4096 x 4608 x 1152 int8 with
// gelu_tanh and residual 25.0 -> 26.4 us.)
template <int BN>
constexpr bool kWide = BN <= 192;
constexpr int kEpBox = 32 * 128;

struct ResStream {
  const CUtensorMap* tmR;  // null: no residual
  uint64_t* bar;           // the box of R has arrived
  uint8_t* box;
  uint32_t issued, used;   // boxes asked for (lane 0) and consumed
};

// Lane 0: asks for R's box at (row0, col0), if it lies inside R.
__device__ __forceinline__ void res_load(const GemmEpParams& p, ResStream& s, int row0, int col0) {
  if (row0 < p.T && col0 < p.N) {
    mbar_arrive_expect_tx(s.bar, kEpBox);
    tma_load_2d(s.box, s.tmR, col0, row0, s.bar);
  } else {
    mbar_arrive(s.bar);  // nothing there: the box is not read
  }
  ++s.issued;
}

// z (chunk c, 0 or 1, of this thread's row) -> R + g * act(z) -> bf16 in the
// warp's box.
__device__ __forceinline__ void epi_box_ep(const GemmEpParams& p, f2 (&z)[16], int c, int col,
                                           const uint16_t* gate_row, bool has_res, uint8_t* box,
                                           int lane) {
  uint4 g[4];
  if (gate_row) {
#pragma unroll
    for (int q = 0; q < 4; ++q)
      g[q] = col + 8 * q < p.N ? *reinterpret_cast<const uint4*>(gate_row + col + 8 * q)
                               : make_uint4(0, 0, 0, 0);
  }
  act_chunk(p.act, z);
  if (gate_row) {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const uint32_t w[4] = {g[q].x, g[q].y, g[q].z, g[q].w};
#pragma unroll
      for (int i = 0; i < 4; ++i) z[4 * q + i] = mul2(z[4 * q + i], unpack_bf16x2(w[i]));
    }
  }
  uint8_t* row = box + lane * 128;
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    uint4* slot = reinterpret_cast<uint4*>(row + (((4 * c + q) ^ (lane & 7)) << 4));
    if (has_res) {
      const uint4 rv = *slot;
      const uint32_t w[4] = {rv.x, rv.y, rv.z, rv.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) z[4 * q + i] = add2(z[4 * q + i], unpack_bf16x2(w[i]));
    }
    *slot = make_uint4(pack_bf16x2(z[4 * q].x, z[4 * q].y),
                       pack_bf16x2(z[4 * q + 1].x, z[4 * q + 1].y),
                       pack_bf16x2(z[4 * q + 2].x, z[4 * q + 2].y),
                       pack_bf16x2(z[4 * q + 3].x, z[4 * q + 3].y));
  }
}

// As epi_tile for the warp's 64 columns, ending in  Y = bf16(R + g * act(z)).
// (next_row0, next_col0): the warp's corner in its next tile, next_row0 < 0 for
// none.  Returns false if a wait gave up.
template <int KIND, int W, int LOGO, class RelAcc, class RelPrm>
__device__ __forceinline__ bool epi_tile_ep(const GemmEpParams& p, const CUtensorMap* tmY,
                                            ResStream& s, uint32_t t_addr, const EpiTile& e,
                                            const uint16_t* gate_row, const float* prm,
                                            int prm_col, int next_row0, int next_col0, int lane,
                                            const WaitCtl& wc, RelAcc release_acc,
                                            RelPrm release_params) {
  static_assert(LOGO == 0 || (LOGO >= 4 && LOGO <= 6), "output blocks of 16, 32 or 64 columns");
  const bool has_res = s.tmR != nullptr;
  // the box: R's has arrived, or the previous tile's store has read it
  if (has_res) {
    const bool got = mbar_wait(s.bar, s.used & 1u, wc);
    if (!__all_sync(0xffffffffu, got)) return false;  // (not used: the caller waits again)
    ++s.used;
  } else {
    if (lane == 0) bulk_wait_group_read<0>();
    __syncwarp();
  }
  if (e.row0 >= p.T || e.col_base >= p.N) {  // nothing of Y here
    release_acc();
    release_params();
  } else if constexpr (LOGO < 6) {
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      uint32_t r[32];
      tmem_ld_32x32b_x32(t_addr + uint32_t(c * 32), r);
      tmem_wait_ld();
      if (c == 1) release_acc();
      f2 z[16];
      if constexpr (KIND == kBF16) {
        epi_z_bf16(r, c, reinterpret_cast<const uint16_t*>(prm) + prm_col, z);
      } else if constexpr (LOGO == 0) {
        epi_z<W>(p, r, c, e, prm + prm_col, z);
      } else {
        epi_dequant<W>(p, r, c, e, prm + prm_col, z);
        fwht_chunk<LOGO>(z);
        epi_finish<W>(p, z, c, prm + prm_col);
      }
      if (c == 1) release_params();
      epi_box_ep(p, z, c, e.col_base + c * 32, gate_row, has_res, s.box, lane);
    }
  } else {
    f2 z[2][16];
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      uint32_t r[32];
      tmem_ld_32x32b_x32(t_addr + uint32_t(c * 32), r);
      tmem_wait_ld();
      if (c == 1) release_acc();
      epi_dequant<W>(p, r, c, e, prm + prm_col, z[c]);
      fwht_chunk<5>(z[c]);
    }
    // index bit 5: between the two 32-column chunks
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const f2 x = z[0][i], y = z[1][i];
      z[0][i] = add2(x, y);
      z[1][i] = sub2(x, y);
    }
#pragma unroll
    for (int c = 0; c < 2; ++c) epi_finish<W>(p, z[c], c, prm + prm_col);
    release_params();
#pragma unroll
    for (int c = 0; c < 2; ++c)
      epi_box_ep(p, z[c], c, e.col_base + c * 32, gate_row, has_res, s.box, lane);
  }
  fence_proxy_async_smem();
  __syncwarp();
  if (lane == 0) {
    if (e.row0 < p.T && e.col_base < p.N) tma_store_2d(tmY, s.box, e.col_base, e.row0);
    bulk_commit_group();
    if (has_res && next_row0 >= 0) {
      bulk_wait_group_read<0>();
      res_load(p, s, next_row0, next_col0);
    }
  }
  return true;
}

// Residual columns [col, col + 32) of `row` (zeros where there are none).
__device__ __forceinline__ void load_residual(const GemmEpParams& p, int64_t row, int col,
                                              uint4 (&v)[4]) {
  if (p.residual == nullptr) return;
  const uint16_t* src = p.residual + row * p.N + col;
#pragma unroll
  for (int q = 0; q < 4; ++q)
    v[q] = row < p.T && col + 8 * q < p.N ? *reinterpret_cast<const uint4*>(src + 8 * q)
                                          : make_uint4(0, 0, 0, 0);
}

// The lean layout: the warp's HC columns in 32-column chunks through one box.
// `res` holds the first chunk's residual on entry and the next tile's (row
// next_row, columns from next_col on; next_row < 0: none) on exit.
template <int KIND, int HC, int W, int LOGO, class RelAcc, class RelPrm>
__device__ __forceinline__ void epi_tile_lean(const GemmEpParams& p, const CUtensorMap* tmY,
                                              uint32_t t_addr, const EpiTile& e,
                                              const uint16_t* gate_row, const float* prm,
                                              int prm_col, uint4 (&res)[4], int64_t next_row,
                                              int next_col, uint8_t* box, int lane,
                                              RelAcc release_acc, RelPrm release_params) {
  constexpr int NCH = HC / 32;
  auto finish = [&](f2 (&z)[16], int c) {
    const int col = e.col_base + c * 32;
    uint4 g[4];
    if (gate_row) {
#pragma unroll
      for (int q = 0; q < 4; ++q)
        g[q] = col + 8 * q < p.N ? *reinterpret_cast<const uint4*>(gate_row + col + 8 * q)
                                 : make_uint4(0, 0, 0, 0);
    }
    act_chunk(p.act, z);
    if (gate_row) {
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const uint32_t w[4] = {g[q].x, g[q].y, g[q].z, g[q].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) z[4 * q + i] = mul2(z[4 * q + i], unpack_bf16x2(w[i]));
      }
    }
    if (p.residual != nullptr) {
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const uint32_t w[4] = {res[q].x, res[q].y, res[q].z, res[q].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) z[4 * q + i] = add2(z[4 * q + i], unpack_bf16x2(w[i]));
      }
      if (c + 1 < NCH)
        load_residual(p, e.row, col + 32, res);
      else if (next_row >= 0)
        load_residual(p, next_row, next_col, res);
    }
    uint32_t packed[16];
    pack_chunk(z, packed);
    if (lane == 0) bulk_wait_group_read<0>();  // the previous chunk's store has read the box
    __syncwarp();
    epi_store_chunk(p, tmY, packed, col, e.row0, box, lane);
  };
  constexpr int G = LOGO == 6 ? 2 : 1;
  // chunks past Y's last column are left out, all of them below its last row
  const int live = e.row0 >= p.T || e.col_base >= p.N ? 0 : (p.N - e.col_base + 31) / 32;
#pragma unroll 1
  for (int c0 = 0; c0 < NCH; c0 += G) {
    if (c0 >= live) {
      // (next tile's residual: the last live chunk has not asked for it)
      if (p.residual != nullptr && next_row >= 0) load_residual(p, next_row, next_col, res);
      release_acc();
      release_params();
      return;
    }
    f2 z[G][16];
#pragma unroll
    for (int c = 0; c < G; ++c) {
      uint32_t r[32];
      tmem_ld_32x32b_x32(t_addr + uint32_t((c0 + c) * 32), r);
      tmem_wait_ld();
      if (c0 + c == NCH - 1) release_acc();
      if constexpr (KIND == kBF16) {
        epi_z_bf16(r, c0 + c, reinterpret_cast<const uint16_t*>(prm) + prm_col, z[c]);
      } else if constexpr (LOGO == 0) {
        epi_z<W>(p, r, c0 + c, e, prm + prm_col, z[c]);
      } else {
        epi_dequant<W>(p, r, c0 + c, e, prm + prm_col, z[c]);
        fwht_chunk<(LOGO < 5 ? LOGO : 5)>(z[c]);
      }
    }
    if constexpr (LOGO == 6) {
      // index bit 5: between the two 32-column chunks
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const f2 x = z[0][i], y = z[1][i];
        z[0][i] = add2(x, y);
        z[1][i] = sub2(x, y);
      }
    }
    if constexpr (LOGO > 0) {
#pragma unroll
      for (int c = 0; c < G; ++c) epi_finish<W>(p, z[c], c0 + c, prm + prm_col);
    }
    if (c0 + G == NCH) release_params();
#pragma unroll
    for (int c = 0; c < G; ++c) finish(z[c], c0 + c);
  }
}

// This thread's row of the gate, or null (no gate, or a row past T).
__device__ __forceinline__ const uint16_t* gate_row_of(const GemmEpParams& p, int64_t row) {
  return p.gate != nullptr && row < p.T ? p.gate + (row / p.gate_rows) * p.N : nullptr;
}

}  // namespace

namespace {

// Arrivals beyond the usual one that a barrier of this kind waits for: one that
// never comes where the test hook asks for it, else none.  (A branch in the
// producer's loop instead cost the pair 3 us of 38.)
template <bool EP>
__device__ __forceinline__ uint32_t withheld(const GemmArgs<EP>& p, int what) {
  if constexpr (EP)
    return p.withhold == what ? 1u : 0u;
  else
    return 0u;
}

// The copies into the last two parameter slots, of `n` in all, have landed.
__device__ __forceinline__ void wait_param_copies(uint64_t* pfull, uint32_t n, const WaitCtl& wc) {
  for (uint32_t j = n > 2 ? n - 2 : 0; j < n; ++j)
    (void)mbar_wait(&pfull[j & 1u], (j >> 1) & 1u, wc);
}

}  // namespace

// ------------------------------------------------------- single-CTA kernel
template <int KIND, int BN, bool PK, bool EP>
struct GemmCfg {
  static constexpr int A_BYTES = PK ? 0 : BM * BK;      // A's shared stage (PK: in tensor memory)
  static constexpr int B_BYTES = BN * BK;
  static constexpr int P_BYTES = PK ? BM * BK / 2 : 0;  // packed A as loaded (64-byte swizzle)
  static constexpr int STAGE_BYTES = A_BYTES + B_BYTES + P_BYTES;
  static constexpr uint32_t STAGE_TX = uint32_t(STAGE_BYTES);  // bytes the tensor loads bring
  static constexpr bool WIDE = EP && kWide<BN>;
  static constexpr int EPW = WIDE ? BN / 16 : kEpiWarps;  // epilogue warps
  static constexpr int THREADS = 64 + 32 * EPW + (PK ? 32 * kConvWarps : 0);
  static constexpr int NBAR_STAGE = PK ? 3 : 2;  // full, empty (, converted)
  static constexpr int HC = BN * 4 / EPW;  // columns per epilogue warp
  // accumulator chunks read per tensor-memory wait: at most 3; one for packed
  // 192-column tiles, whose 448 threads leave 128 registers a thread
  static constexpr int EPI_GMAX = (PK && BN == 192) ? 1 : 3;
  static constexpr int NBOX = 1;  // output staging boxes per epilogue warp
  static constexpr int EPI_STAGE_BYTES = WIDE ? kEpBox : NBOX * kStageBox;
  static constexpr int RING_BYTES = 2 * 3 * BN * 4;
  static constexpr int RES_BAR_BYTES = WIDE ? 8 * EPW : 0;
  static constexpr int CTL_BYTES = 256 + RES_BAR_BYTES;
  static constexpr int FIXED = EPW * EPI_STAGE_BYTES + RING_BYTES + CTL_BYTES + 1024;
  static constexpr int STAGES_RAW = (kSmemLimit - FIXED) / STAGE_BYTES;
  // PK: A's stages (32 columns each) follow the two accumulators in the 512
  // columns of tensor memory; the barrier block holds 7 stages of 3 barriers
  static constexpr int TMEM_STAGE_CAP = PK ? (512 - 2 * BN) / 32 : 8;
  static constexpr int STAGE_CAP = PK ? (TMEM_STAGE_CAP < 7 ? TMEM_STAGE_CAP : 7) : 8;
  static constexpr int STAGES = STAGES_RAW > STAGE_CAP ? STAGE_CAP : STAGES_RAW;
  static constexpr int A_COL0 = 2 * BN;  // first tensor-memory column of A's stages (PK)
  static constexpr int TMEM_COLS = tmem_cols_for(2 * BN + (PK ? 32 * STAGES : 0));
  static constexpr uint32_t IDESC = KIND == kBF16 ? bf16_idesc(BM, BN) : i8_idesc(BM, BN);
  static constexpr size_t SMEM = size_t(STAGES) * STAGE_BYTES + FIXED;
  static_assert(BN % 64 == 0 && BN >= 64 && BN <= 256, "two 32-column-aligned halves");
  static_assert(B_BYTES % 1024 == 0, "stage bases must stay 1024-byte aligned");
  static_assert(STAGES >= 2, "shared / tensor memory budget");
  static_assert(!PK || 2 * BN + 32 * STAGES <= 512, "tensor memory budget");
  static_assert(8 * NBAR_STAGE * STAGES + 88 + RES_BAR_BYTES <= CTL_BYTES, "barrier block");
  static_assert(KIND == kI8 || !PK, "packed codes are integers");
  static_assert(SMEM <= size_t(kSmemLimit), "shared memory budget");
};

// tmR: the residual's tensor map, or null (always null without EP).
template <int KIND, int BN, int LOGO, bool PK, bool EP>
__device__ __forceinline__ void gemm_body(const CUtensorMap* tmA, const CUtensorMap* tmB,
                                          const CUtensorMap* tmY, const CUtensorMap* tmR,
                                          const GemmArgs<EP>& p) {
  using C = GemmCfg<KIND, BN, PK, EP>;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_addr = smem_u32(smem_raw);
  uint8_t* smem = smem_raw + (((raw_addr + 1023u) & ~1023u) - raw_addr);
  uint8_t* sA = smem;
  uint8_t* sB = smem + size_t(C::STAGES) * C::A_BYTES;
  uint8_t* sP = sB + size_t(C::STAGES) * C::B_BYTES;  // packed A (PK only)
  uint8_t* epi_stage = sP + size_t(C::STAGES) * C::P_BYTES;  // 1024-aligned
  float* ring = reinterpret_cast<float*>(epi_stage + C::EPW * C::EPI_STAGE_BYTES);
  uint64_t* full = reinterpret_cast<uint64_t*>(reinterpret_cast<uint8_t*>(ring) + C::RING_BYTES);
  uint64_t* empty = full + C::STAGES;
  uint64_t* conv = empty + C::STAGES;    // (PK) stage s's A widened into tensor memory
  uint64_t* tfull = conv + (PK ? C::STAGES : 0);  // [2] accumulator complete
  uint64_t* tempty = tfull + 2;          // [2] accumulator drained by the epilogue
  uint64_t* pfull = tempty + 2;          // [2] parameter slot loaded
  uint64_t* pempty = pfull + 2;          // [2] parameter slot read by the epilogue
  uint64_t* drain = pempty + 2;
  uint64_t* rbar = drain + 1;  // [EPW] box of the residual arrived (wide epilogue)
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(rbar + (C::WIDE ? C::EPW : 0));
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  uint32_t* issued_by = tmem_slot + 2;  // [2]: stages and parameter slots loaded

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const WaitCtl wc{p.err, p.wait_ns};

  param_ring_zero<BN>(ring, threadIdx.x, C::THREADS);
  fence_proxy_async_smem();  // the zeros precede the ring's bulk copies
  if (threadIdx.x == 0) {
    for (int s = 0; s < C::STAGES; ++s) {
      mbar_init(&full[s], 1 + (s == 0 ? withheld<EP>(p, kWithholdStage) : 0u));
      mbar_init(&empty[s], 1);
      if (PK) mbar_init(&conv[s], kConvWarps);  // one arrival per converter warp
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(&tfull[a], 1);
      mbar_init(&tempty[a], C::EPW);  // one arrival per epilogue warp
      mbar_init(&pfull[a], 1);
      mbar_init(&pempty[a], C::EPW);
    }
    mbar_init(drain, 1);
    if constexpr (C::WIDE)
      for (int i = 0; i < C::EPW; ++i)
        mbar_init(&rbar[i], 1 + withheld<EP>(p, kWithholdResidual));
    *abort_flag = 0;
    fence_mbarrier_init();
    prefetch_tmap(tmA);
    prefetch_tmap(tmB);
    prefetch_tmap(tmY);
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, C::TMEM_COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;

  const int num_tiles = p.num_m_tiles * p.num_n_tiles;
  const int KB = (p.K + BK - 1) / BK;

  if (warp == 0) {
    if (lane == 0) {
      // ---------------------------------------------------------- producer
      int stage = 0;
      uint32_t phase = 0;
      int issued = 0, tiles_issued = 0;
      bool ok = true;
      for (int tile = blockIdx.x; tile < num_tiles && ok; tile += gridDim.x) {
        const int m_idx = tile_m(p, tile);
        const int n_idx = tile_n(p, tile);
        const int a = tiles_issued & 1;
        if (*abort_flag || !mbar_wait(&pempty[a], ((tiles_issued >> 1) & 1) ^ 1u, wc)) {
          *abort_flag = 1;
          ok = false;
          break;
        }
        if constexpr (KIND == kBF16)
          param_ring_load16<BN>(p, ring + a * 3 * BN, n_idx * BN, &pfull[a]);
        else
          param_ring_load<BN>(p, ring + a * 3 * BN, n_idx * BN, &pfull[a]);
        ++tiles_issued;
        for (int kb = 0; kb < KB; ++kb) {
          if (*abort_flag || !mbar_wait(&empty[stage], phase ^ 1u, wc)) {
            *abort_flag = 1;
            ok = false;
            break;
          }
          mbar_arrive_expect_tx(&full[stage], C::STAGE_TX);
          if constexpr (PK)  // K bytes of packed A per stage: BK / 2 (a multiple of 16)
            tma_load_2d(sP + size_t(stage) * C::P_BYTES, tmA, kb * (BK / 2), m_idx * BM,
                        &full[stage]);
          else
            tma_load_2d(sA + size_t(stage) * C::A_BYTES, tmA, kb * BK, m_idx * BM, &full[stage]);
          tma_load_2d(sB + size_t(stage) * C::B_BYTES, tmB, kb * BK, n_idx * BN, &full[stage]);
          ++issued;
          if (++stage == C::STAGES) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
      issued_by[0] = uint32_t(issued);
      issued_by[1] = uint32_t(tiles_issued);
    }
  } else if (warp == 1) {
    // --------------------------------------------------------- MMA issuer
    // The warp runs the loop converged and one elected thread issues: issued
    // from inside one lane's branch the loop itself (barrier tests, descriptors,
    // commits) was in the MMAs' way where a tile has few K blocks (256 x 1024 x
    // 1024 int8 6.2 -> 5.5 us, 16384 x 4096 x 8192 349 -> 335 us).
    int stage = 0;
    uint32_t phase = 0;
    int acc_iter = 0;
    bool ok = true;
    const bool leader = elect_one();
    const uint64_t a_desc0 = sw128_kmajor_desc(smem_u32(sA));
    const uint64_t b_desc0 = sw128_kmajor_desc(smem_u32(sB));
    for (int tile = blockIdx.x; tile < num_tiles && ok; tile += gridDim.x, ++acc_iter) {
      const int acc = acc_iter & 1;
      const uint32_t acc_phase = (acc_iter >> 1) & 1;
      if (!__all_sync(0xffffffffu,
                      !*abort_flag && mbar_wait(&tempty[acc], acc_phase ^ 1u, wc))) {
        *abort_flag = 1;
        break;
      }
      tc_fence_after();
      const uint32_t d_tmem = tmem_base + uint32_t(acc * BN);
      for (int kb = 0; kb < KB; ++kb) {
        // B landed (full) and, for packed A, the converters stored A (conv)
        if (!__all_sync(0xffffffffu, mbar_wait(&full[stage], phase, wc) &&
                                         (!PK || mbar_wait(&conv[stage], phase, wc)))) {
          *abort_flag = 1;
          ok = false;
          break;
        }
        tc_fence_after();
        if (leader) {
          const uint64_t adesc = a_desc0 + uint64_t(stage) * (C::A_BYTES >> 4);
          const uint64_t bdesc = b_desc0 + uint64_t(stage) * (C::B_BYTES >> 4);
#pragma unroll
          for (int k = 0; k < BK / 32; ++k) {
            // advance 32 bytes along K inside the swizzle row (encoded >> 4)
            if constexpr (PK)  // A in tensor memory: 8 columns of four codes per 32 bytes
              mma_i8_tmem_a(d_tmem, tmem_base + uint32_t(C::A_COL0 + 32 * stage + 8 * k),
                            bdesc + uint64_t(2 * k), C::IDESC, (kb > 0 || k > 0) ? 1u : 0u);
            else
              mma_kind<KIND>(d_tmem, adesc + uint64_t(2 * k), bdesc + uint64_t(2 * k), C::IDESC,
                             (kb > 0 || k > 0) ? 1u : 0u);
          }
          mma_commit(&empty[stage]);
          if (kb + 1 == KB) mma_commit(&tfull[acc]);
        }
        __syncwarp();
        if (++stage == C::STAGES) {
          stage = 0;
          phase ^= 1u;
        }
      }
    }
    // wait for every issued MMA before tensor memory can be released
    if (leader) mma_commit(drain);
    __syncwarp();
    (void)mbar_wait(drain, 0, wc);
    __syncwarp();
  } else if (warp < 2 + C::EPW) {
    // ----------------------------------------------------------- epilogue
    const int ew = warp - 2;         // 0 .. EPW - 1
    const int quarter = warp & 3;    // TMEM lanes [32*quarter, 32*quarter + 32)
    const int half = ew >> 2;        // columns [half*HC, half*HC + HC) of the tile
    uint8_t* stg = epi_stage + ew * C::EPI_STAGE_BYTES;
    [[maybe_unused]] ResStream rs{tmR, rbar + ew, stg, 0, 0};
    int acc_iter = 0;
    float sx_next = 0.0f, mt_next = 0.0f;
    if (KIND == kI8 && int(blockIdx.x) < num_tiles)
      load_row_params(p, int64_t(tile_m(p, int(blockIdx.x))) * BM + quarter * 32 + lane,
                      sx_next, mt_next);
    [[maybe_unused]] uint4 res[4];
    if constexpr (EP && !C::WIDE) {
      if (int(blockIdx.x) < num_tiles)
        load_residual(p, int64_t(tile_m(p, int(blockIdx.x))) * BM + quarter * 32 + lane,
                      tile_n(p, int(blockIdx.x)) * BN + half * C::HC, res);
    }
    if constexpr (C::WIDE) {
      if (tmR && lane == 0 && int(blockIdx.x) < num_tiles)
        res_load(p, rs, tile_m(p, int(blockIdx.x)) * BM + quarter * 32,
                 tile_n(p, int(blockIdx.x)) * BN + half * C::HC);
    }
    for (int tile = blockIdx.x; tile < num_tiles; tile += gridDim.x, ++acc_iter) {
      const int acc = acc_iter & 1;
      const uint32_t acc_phase = (acc_iter >> 1) & 1;
      const int m_idx = tile_m(p, tile);
      const int n_idx = tile_n(p, tile);
      EpiTile e;
      e.row0 = m_idx * BM + quarter * 32;
      e.col_base = n_idx * BN + half * C::HC;
      e.row = int64_t(e.row0) + lane;
      e.row_ok = e.row < p.T;
      e.sx = sx_next;
      e.mt = mt_next;
      const int next = tile + int(gridDim.x);
      if (KIND == kI8 && next < num_tiles)  // next tile's row parameters, in flight during this one
        load_row_params(p, int64_t(tile_m(p, next)) * BM + quarter * 32 + lane, sx_next,
                        mt_next);
      const bool got = !(*abort_flag) && mbar_wait(&tfull[acc], acc_phase, wc) &&
                       mbar_wait(&pfull[acc], acc_phase, wc);
      if (!__all_sync(0xffffffffu, got)) {
        *abort_flag = 1;
        break;
      }
      tc_fence_after();
      const uint32_t t_addr = tmem_base + uint32_t(acc * BN + half * C::HC) +
                              (uint32_t(quarter * 32) << 16);
      auto release_acc = [&] {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&tempty[acc]);
      };
      auto release_params = [&] {
        // the parameter reads (generic proxy), each thread's ordered
        // before the next bulk copy into the slot by its proxy fence
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&pempty[acc]);
      };
      if constexpr (EP) {
        const int next_row0 = next < num_tiles ? tile_m(p, next) * BM + quarter * 32 : -1;
        const int next_col0 = next < num_tiles ? tile_n(p, next) * BN + half * C::HC : 0;
        if constexpr (C::WIDE) {
          if (!epi_tile_ep<KIND, BN, LOGO>(p, tmY, rs, t_addr, e, gate_row_of(p, e.row),
                                           ring + acc * 3 * BN, half * C::HC, next_row0, next_col0,
                                           lane, wc, release_acc, release_params)) {
            *abort_flag = 1;
            break;
          }
        } else {
          epi_tile_lean<KIND, C::HC, BN, LOGO>(
              p, tmY, t_addr, e, gate_row_of(p, e.row), ring + acc * 3 * BN, half * C::HC, res,
              next_row0 < 0 ? -1 : int64_t(next_row0) + lane, next_col0, stg, lane, release_acc,
              release_params);
        }
      } else {
        epi_tile<C::HC, BN, C::NBOX, LOGO, C::EPI_GMAX>(
            p, tmY, t_addr, e, ring + acc * 3 * BN + half * C::HC, stg, lane, release_acc,
            release_params);
      }
    }
    if constexpr (C::WIDE) {
      if (tmR && lane == 0 && rs.used < rs.issued)  // after a give-up: the box in flight lands
        (void)mbar_wait(rs.bar, rs.used & 1u, wc);
    }
    if (lane == 0) bulk_wait_group<0>();  // all of this warp's stores are complete
    __syncwarp();
  } else if constexpr (PK) {
    // ------------------------------------------------- packed-A converters
    // Lane i of converter warp w owns row r = 32 (w % 4) + i of every A tile,
    // which is tensor-memory lane r.  Per stage it reads the row's 64 packed
    // bytes (four 16-byte chunks; with the 64-byte swizzle chunk c of row r
    // sits at chunk c ^ ((r >> 1) & 3), so the 8 rows of a quarter-warp read
    // 8 distinct bank groups), widens them to 128 int8 values and stores
    // them as 32 columns of four values each at A's stage in tensor memory.
    const int quarter = warp & 3;
    const int r = quarter * 32 + lane;
    const int swz = (r >> 1) & 3;
    const uint32_t t_row = tmem_base + (uint32_t(quarter * 32) << 16) + uint32_t(C::A_COL0);
    int stage = 0;
    uint32_t phase = 0;
    bool ok = true;
    for (int tile = blockIdx.x; tile < num_tiles && ok; tile += gridDim.x) {
      for (int kb = 0; kb < KB; ++kb) {
        // the stage's packed tile has landed, and the MMAs that read its
        // previous A from tensor memory have completed
        const bool got = !(*abort_flag) && mbar_wait(&full[stage], phase, wc) &&
                         mbar_wait(&empty[stage], phase ^ 1u, wc);
        if (!__all_sync(0xffffffffu, got)) {
          *abort_flag = 1;
          ok = false;
          break;
        }
        tc_fence_after();
        const uint8_t* src = sP + size_t(stage) * C::P_BYTES + r * 64;
        uint32_t a[32];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const uint4 v = *reinterpret_cast<const uint4*>(src + ((c ^ swz) << 4));
          widen_i4x8(v.x, a[8 * c + 0], a[8 * c + 1]);
          widen_i4x8(v.y, a[8 * c + 2], a[8 * c + 3]);
          widen_i4x8(v.z, a[8 * c + 4], a[8 * c + 5]);
          widen_i4x8(v.w, a[8 * c + 6], a[8 * c + 7]);
        }
        tmem_st_32x32b_x32(t_row + uint32_t(32 * stage), a);
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&conv[stage]);
        if (++stage == C::STAGES) {
          stage = 0;
          phase ^= 1u;
        }
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  // after a give-up, whoever gave up, the copies in flight land before the CTA
  // can exit
  if (*abort_flag && threadIdx.x == 0) {
    const int n = int(issued_by[0]);
    for (int i = n > C::STAGES ? n - C::STAGES : 0; i < n; ++i)
      (void)mbar_wait(&full[i % C::STAGES], uint32_t(i / C::STAGES) & 1u, wc);
    wait_param_copies(pfull, issued_by[1], wc);
  }
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem_base, C::TMEM_COLS);
  }
}

// ---------------------------------------------------------- CTA-pair kernel
// BN: output columns per pair tile (N of each MMA); 256 without EP.
template <int KIND, int BN, bool EP>
struct PairCfg {
  static constexpr int BM_PAIR = 2 * BM;  // output rows per pair tile (M of each MMA)
  static constexpr int B_ROWS = BN / 2;   // rows of B each CTA holds
  static constexpr int A_BYTES = BM * BK;
  static constexpr int B_BYTES = B_ROWS * BK;
  static constexpr int STAGE_BYTES = A_BYTES + B_BYTES;  // per CTA
  static constexpr bool WIDE = EP && kWide<BN>;
  static constexpr int EPW = WIDE ? BN / 16 : kEpiWarps;  // epilogue warps
  static constexpr int THREADS = 64 + 32 * EPW;
  static constexpr int HC = BN * 4 / EPW;  // columns per epilogue warp
  static constexpr int NBOX = EP ? 1 : 2;  // output staging boxes per epilogue warp
  static constexpr int EPI_STAGE_BYTES = WIDE ? kEpBox : NBOX * kStageBox;
  static constexpr int RES_BAR_BYTES = WIDE ? 8 * EPW : 0;
  static constexpr int RING_BYTES = 2 * 3 * BN * 4;
  static constexpr int CTL_BYTES = 512;
  static constexpr int FIXED = EPW * EPI_STAGE_BYTES + RING_BYTES + CTL_BYTES + 1024;
  static constexpr int STAGES_RAW = (kSmemLimit - FIXED) / STAGE_BYTES;
  static constexpr int STAGES = STAGES_RAW > 8 ? 8 : STAGES_RAW;
  static constexpr int TMEM_COLS = tmem_cols_for(2 * BN);
  static constexpr uint32_t IDESC =
      KIND == kBF16 ? bf16_idesc(BM_PAIR, BN) : i8_idesc(BM_PAIR, BN);
  static constexpr size_t SMEM = size_t(STAGES) * STAGE_BYTES + FIXED;
  static_assert(B_BYTES % 1024 == 0, "stage bases must stay 1024-byte aligned");
  static_assert(STAGES >= 2, "shared memory budget");
  static_assert(16 * STAGES + 96 + RES_BAR_BYTES <= CTL_BYTES, "barrier block");
  static_assert(SMEM <= size_t(kSmemLimit), "shared memory budget");
};

// Clusters of two CTAs; CTA rank r of a cluster owns rows [128 r, 128 r + 128)
// of every 256-row pair tile (its A rows and its half of the accumulator) and
// B rows [128 r, 128 r + 128) of the tile's 256 columns.  Barriers, all in
// each CTA's own shared memory (those marked "rank 0" used only there):
//   full[s]    (rank 0) stage s of both CTAs landed: rank 0's producer
//              expects the bytes of both and both CTAs' copies count on it;
//   empty[s]   the MMAs have read stage s (pair commit to both CTAs);
//   tfull[a]   accumulator a is complete (pair commit to both CTAs);
//   tempty[a]  (rank 0) the 16 epilogue warps of the pair have read
//              accumulator a (remote arrivals);
//   pfull[a], pempty[a]   this CTA's parameter slot a loaded / read;
//   drain      every MMA issued has completed (pair commit to both CTAs).
// At exit each producer posts the number of stages it loaded to rank 0,
// whose producer then waits until every copy of either CTA has landed: it
// supplies the missing arrival or cancels the missing bytes of a stage that
// only one CTA loaded (after a bounded wait gave up).
// tmR: the residual's tensor map, or null (always null without the wide epilogue).
template <int KIND, int BN, bool EP>
__device__ __forceinline__ void gemm_pair_body(const CUtensorMap* tmA, const CUtensorMap* tmB,
                                               const CUtensorMap* tmY, const CUtensorMap* tmR,
                                               const GemmArgs<EP>& p) {
  using C = PairCfg<KIND, BN, EP>;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_addr = smem_u32(smem_raw);
  uint8_t* smem = smem_raw + (((raw_addr + 1023u) & ~1023u) - raw_addr);
  uint8_t* sA = smem;
  uint8_t* sB = smem + size_t(C::STAGES) * C::A_BYTES;
  uint8_t* epi_stage = sB + size_t(C::STAGES) * C::B_BYTES;  // 1024-aligned
  float* ring = reinterpret_cast<float*>(epi_stage + C::EPW * C::EPI_STAGE_BYTES);
  uint64_t* full = reinterpret_cast<uint64_t*>(reinterpret_cast<uint8_t*>(ring) + C::RING_BYTES);
  uint64_t* empty = full + C::STAGES;
  uint64_t* tfull = empty + C::STAGES;
  uint64_t* tempty = tfull + 2;
  uint64_t* pfull = tempty + 2;
  uint64_t* pempty = pfull + 2;
  uint64_t* drain = pempty + 2;
  uint64_t* rbar = drain + 1;  // [EPW] box of the residual arrived (wide epilogue)
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(rbar + (C::WIDE ? C::EPW : 0));
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  // [0], [1] (rank 0): stages each CTA loaded; [2]: parameter slots this CTA loaded
  uint32_t* issued_by = tmem_slot + 2;

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const WaitCtl wc{p.err, p.wait_ns};

  param_ring_zero<BN>(ring, threadIdx.x, C::THREADS);
  fence_proxy_async_smem();  // the zeros precede the ring's bulk copies
  if (threadIdx.x == 0) {
    for (int s = 0; s < C::STAGES; ++s) {
      mbar_init(&full[s], 1 + (s == 0 ? withheld<EP>(p, kWithholdStage) : 0u));
      mbar_init(&empty[s], 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(&tfull[a], 1);
      mbar_init(&tempty[a], 2 * C::EPW);
      mbar_init(&pfull[a], 1);
      mbar_init(&pempty[a], C::EPW);
    }
    mbar_init(drain, 1);
    if constexpr (C::WIDE)
      for (int i = 0; i < C::EPW; ++i)
        mbar_init(&rbar[i], 1 + withheld<EP>(p, kWithholdResidual));
    *abort_flag = 0;
    issued_by[0] = issued_by[1] = 0;
    fence_mbarrier_init();
    prefetch_tmap(tmA);
    prefetch_tmap(tmB);
    prefetch_tmap(tmY);
  }
  if (warp == 1) {
    tmem_alloc_pair(tmem_slot, C::TMEM_COLS);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // both CTAs' barriers initialised and tensor memory allocated
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;

  const int num_tiles = p.num_m_tiles * p.num_n_tiles;
  const int cluster_id = int(blockIdx.x >> 1);
  const int num_clusters = int(gridDim.x >> 1);
  const int KB = (p.K + BK - 1) / BK;

  if (warp == 0) {
    if (lane == 0) {
      // ---------------------------------------------------------- producer
      const uint32_t full0 = mapa_shared(full, 0);  // rank 0's full[0]
      int stage = 0;
      uint32_t phase = 0;
      int issued = 0, tiles_issued = 0;
      bool ok = true;
      for (int tile = cluster_id; tile < num_tiles && ok; tile += num_clusters) {
        const int m_idx = tile_m(p, tile);
        const int n_idx = tile_n(p, tile);
        const int a_row = m_idx * C::BM_PAIR + int(rank) * BM;
        const int b_row = n_idx * BN + int(rank) * C::B_ROWS;
        const int a = tiles_issued & 1;
        if (*abort_flag || !mbar_wait(&pempty[a], ((tiles_issued >> 1) & 1) ^ 1u, wc)) {
          *abort_flag = 1;
          ok = false;
          break;
        }
        if constexpr (KIND == kBF16)
          param_ring_load16<BN>(p, ring + a * 3 * BN, n_idx * BN, &pfull[a]);
        else
          param_ring_load<BN>(p, ring + a * 3 * BN, n_idx * BN, &pfull[a]);
        ++tiles_issued;
        for (int kb = 0; kb < KB; ++kb) {
          if (*abort_flag || !mbar_wait<true>(&empty[stage], phase ^ 1u, wc)) {
            *abort_flag = 1;
            ok = false;
            break;
          }
          if (rank == 0) mbar_arrive_expect_tx(&full[stage], 2 * C::STAGE_BYTES);
          const uint32_t bar = full0 + uint32_t(stage) * 8u;
          tma_load_2d_pair(sA + size_t(stage) * C::A_BYTES, tmA, kb * BK, a_row, bar);
          tma_load_2d_pair(sB + size_t(stage) * C::B_BYTES, tmB, kb * BK, b_row, bar);
          ++issued;
          if (++stage == C::STAGES) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
      issued_by[2] = uint32_t(tiles_issued);
      st_shared_cluster_u32(mapa_shared(&issued_by[rank], 0), uint32_t(issued));
    }
  } else if (warp == 1) {
    if (rank == 0) {
      // ------------------------------------------------ MMA issuer (rank 0)
      // converged, one elected thread issues (see gemm_body)
      int stage = 0;
      uint32_t phase = 0;
      int acc_iter = 0;
      bool ok = true;
      const bool leader = elect_one();
      const uint64_t a_desc0 = sw128_kmajor_desc(smem_u32(sA));
      const uint64_t b_desc0 = sw128_kmajor_desc(smem_u32(sB));
      for (int tile = cluster_id; tile < num_tiles && ok; tile += num_clusters, ++acc_iter) {
        const int acc = acc_iter & 1;
        const uint32_t acc_phase = (acc_iter >> 1) & 1;
        if (!__all_sync(0xffffffffu,
                        !*abort_flag && mbar_wait<true>(&tempty[acc], acc_phase ^ 1u, wc))) {
          *abort_flag = 1;
          break;
        }
        tc_fence_after();
        const uint32_t d_tmem = tmem_base + uint32_t(acc * BN);
        for (int kb = 0; kb < KB; ++kb) {
          if (!__all_sync(0xffffffffu, mbar_wait<true>(&full[stage], phase, wc))) {
            *abort_flag = 1;
            ok = false;
            break;
          }
          tc_fence_after();
          if (leader) {
            const uint64_t adesc = a_desc0 + uint64_t(stage) * (C::A_BYTES >> 4);
            const uint64_t bdesc = b_desc0 + uint64_t(stage) * (C::B_BYTES >> 4);
#pragma unroll
            for (int k = 0; k < BK / 32; ++k) {
              // advance 32 bytes along K inside the swizzle row (encoded >> 4)
              mma_kind_pair<KIND>(d_tmem, adesc + uint64_t(2 * k), bdesc + uint64_t(2 * k),
                                  C::IDESC, (kb > 0 || k > 0) ? 1u : 0u);
            }
            mma_commit_pair(&empty[stage], 0x3);
            if (kb + 1 == KB) mma_commit_pair(&tfull[acc], 0x3);
          }
          __syncwarp();
          if (++stage == C::STAGES) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
      // every issued MMA completes before either CTA releases its shared
      // memory or tensor memory
      if (leader) mma_commit_pair(drain, 0x3);
      __syncwarp();
    }
    // (rank 1: the pair's last commit has landed)
    (void)mbar_wait<true>(drain, 0, wc);
    __syncwarp();
  } else {
    // ----------------------------------------------------------- epilogue
    const int ew = warp - 2;         // 0 .. EPW - 1
    const int quarter = warp & 3;    // TMEM lanes [32*quarter, 32*quarter + 32)
    const int half = ew >> 2;        // columns [half*HC, half*HC + HC) of the tile
    uint8_t* stg = epi_stage + ew * C::EPI_STAGE_BYTES;
    [[maybe_unused]] ResStream rs{tmR, rbar + ew, stg, 0, 0};
    const uint32_t tempty0 = mapa_shared(tempty, 0);
    const int row_off = int(rank) * BM + quarter * 32 + lane;
    int acc_iter = 0;
    float sx_next = 0.0f, mt_next = 0.0f;
    if (KIND == kI8 && cluster_id < num_tiles)
      load_row_params(p, int64_t(tile_m(p, cluster_id)) * C::BM_PAIR + row_off, sx_next,
                      mt_next);
    [[maybe_unused]] uint4 res[4];
    if constexpr (C::WIDE) {
      if (tmR && lane == 0 && cluster_id < num_tiles)
        res_load(p, rs, tile_m(p, cluster_id) * C::BM_PAIR + int(rank) * BM + quarter * 32,
                 tile_n(p, cluster_id) * BN + half * C::HC);
    }
    if constexpr (EP && !C::WIDE) {
      if (cluster_id < num_tiles)
        load_residual(p, int64_t(tile_m(p, cluster_id)) * C::BM_PAIR + row_off,
                      tile_n(p, cluster_id) * BN + half * C::HC, res);
    }
    for (int tile = cluster_id; tile < num_tiles; tile += num_clusters, ++acc_iter) {
      const int acc = acc_iter & 1;
      const uint32_t acc_phase = (acc_iter >> 1) & 1;
      const int m_idx = tile_m(p, tile);
      const int n_idx = tile_n(p, tile);
      EpiTile e;
      e.row0 = m_idx * C::BM_PAIR + int(rank) * BM + quarter * 32;
      e.col_base = n_idx * BN + half * C::HC;
      e.row = int64_t(e.row0) + lane;
      e.row_ok = e.row < p.T;
      e.sx = sx_next;
      e.mt = mt_next;
      const int next = tile + num_clusters;
      if (KIND == kI8 && next < num_tiles)  // next tile's row parameters, in flight during this one
        load_row_params(p, int64_t(tile_m(p, next)) * C::BM_PAIR + row_off, sx_next,
                        mt_next);
      const bool got = !(*abort_flag) && mbar_wait<true>(&tfull[acc], acc_phase, wc) &&
                       mbar_wait(&pfull[acc], acc_phase, wc);
      if (!__all_sync(0xffffffffu, got)) {
        *abort_flag = 1;
        break;
      }
      tc_fence_after();
      const uint32_t t_addr = tmem_base + uint32_t(acc * BN + half * C::HC) +
                              (uint32_t(quarter * 32) << 16);
      auto release_acc = [&] {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_remote(tempty0 + uint32_t(acc) * 8u);
      };
      auto release_params = [&] {
        // the parameter reads (generic proxy), each thread's ordered
        // before the next bulk copy into the slot by its proxy fence
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&pempty[acc]);
      };
      if constexpr (EP) {
        const int next_row0 =
            next < num_tiles ? tile_m(p, next) * C::BM_PAIR + int(rank) * BM + quarter * 32 : -1;
        const int next_col0 = next < num_tiles ? tile_n(p, next) * BN + half * C::HC : 0;
        if constexpr (C::WIDE) {
          if (!epi_tile_ep<KIND, BN, 0>(p, tmY, rs, t_addr, e, gate_row_of(p, e.row),
                                        ring + acc * 3 * BN, half * C::HC, next_row0, next_col0,
                                        lane, wc, release_acc, release_params)) {
            *abort_flag = 1;
            break;
          }
        } else {
          epi_tile_lean<KIND, C::HC, BN, 0>(
              p, tmY, t_addr, e, gate_row_of(p, e.row), ring + acc * 3 * BN, half * C::HC, res,
              next_row0 < 0 ? -1 : int64_t(next_row0) + lane, next_col0, stg, lane, release_acc,
              release_params);
        }
      } else {
        epi_tile<C::HC, BN, C::NBOX, 0, 3>(p, tmY, t_addr, e,
                                              ring + acc * 3 * BN + half * C::HC, stg, lane,
                                              release_acc, release_params);
      }
    }
    if constexpr (C::WIDE) {
      if (tmR && lane == 0 && rs.used < rs.issued)  // after a give-up: the box in flight lands
        (void)mbar_wait(rs.bar, rs.used & 1u, wc);
    }
    if (lane == 0) bulk_wait_group<0>();  // all of this warp's stores are complete
    __syncwarp();
  }

  tc_fence_before();
  __syncthreads();
  cluster_sync();  // both producers have posted their stage counts
  // after a give-up, whoever gave up, the parameter copies in flight land too
  if (*abort_flag && threadIdx.x == 32) wait_param_copies(pfull, issued_by[2], wc);
  if (rank == 0 && threadIdx.x == 0) {
    // every stage copy of either CTA lands before either CTA can exit
    const int L = int(issued_by[0]), P = int(issued_by[1]);
    const int hi = L > P ? L : P;
    for (int s = 0; s < C::STAGES && s < hi; ++s) {
      const int i = s + ((hi - 1 - s) / C::STAGES) * C::STAGES;  // last copy into stage s
      const bool by0 = i < L, by1 = i < P;
      if (by0 && !by1) mbar_complete_tx(&full[s], C::STAGE_BYTES);
      if (by1 && !by0) mbar_arrive_expect_tx(&full[s], C::STAGE_BYTES);
      (void)mbar_wait<true>(&full[s], uint32_t(i / C::STAGES) & 1u, wc);
    }
  }
  __syncthreads();
  cluster_sync();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem_base, C::TMEM_COLS);
  }
}

}  // namespace hq
