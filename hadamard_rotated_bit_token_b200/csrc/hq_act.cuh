// hq_act.cuh -- the activations of the fused epilogues and of the group norm,
// in fp32 on pairs of values, and bf16 pair packing.
//
// silu and both gelus are z * sigmoid(u(z)) with sigmoid(u) = 1 / (1 + 2^(-u log2 e)).
// The special-function units (four lanes a cycle on each quarter of an SM) are
// among what bounds short main loops' epilogues, so two values share one
// reciprocal: with d = 1 + 2^t of each, r = 1 / (d1 d2) gives 1 / d1 = r d2 and
// 1 / d2 = r d1, three special instructions for two values instead of four
// (hq_linear_ep 8192 x 1152 -> 4608 int4 with gelu: 60.6 -> 55.5 us; group norm
// with silu over 16 images of 4096 x 320: 31.9 -> 31.4 us; d1 d2 adds two
// roundings of 2^-24.  Newton steps on the FMA pipe instead of the reciprocal
// made that 26.1 -> 28.4 us: issue slots are as scarce).  The product must not
// overflow, so z enters no lower than where t reaches 63.5; there |z sigmoid(u)|
// is below 4e-18, and any z below returns that or 0 (its value lies between the
// two).  From d1 d2 = 2^126 on the reciprocal is subnormal and flushed, and both
// values come out 0: with t <= 63.5 that takes t >= 62.5 of both, where silu's
// value is at most 43.4 2^-62.5 = 6.6e-18 (gelu_tanh stays below, t <= 62.7).
//   silu       u = z                                                z >= -44
//   gelu_tanh  0.5 (1 + tanh v) = sigmoid(2 v), so
//              u = 2 sqrt(2/pi) (z + 0.044715 z^3)                   z >= -7.6
//   gelu       u = log(Phi(z) / Phi(-z)), an odd function of z: z P(z^2) with P
//              of degree 8, a least-squares fit reweighted towards the largest
//              deviation of u over |z| <= 5.5.  |u| is then off by at most
//              1.4e-5 in fp32, so Phi is within 1.4e-5 of its value relative
//              to itself, on both sides.  Beyond 5.5 P stays at its end
//              value: u grows linearly and z Phi(z) < 1.1e-7 in magnitude on
//              the negative side, as is what the formula gives there; z >= -13.5
// Errors, relative to the value: exponential 2^-22, reciprocal 2^-23, four roundings
// of 2^-24, and t's own, |u| 2^-23 for silu and |u| 2^-22 for gelu_tanh (products and
// rounded constants on the way to t): at most 2^-20 (1 + |u| / 4) in all, 2^-19 at z =
// -44 and 2^-17.5 at -7.6 from t alone.
// relu keeps a NaN (the comparison is false).
#pragma once

#include <cuda_bf16.h>

#include <cstdint>
#include <type_traits>

#include "hq_device.cuh"

namespace hq {

constexpr int kActNone = 0, kActRelu = 1, kActSilu = 2, kActGelu = 3, kActGeluTanh = 4;

__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi) {
  __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&v);
}

__device__ __forceinline__ f2 unpack_bf16x2(uint32_t v) {
  return pk(__uint_as_float(v << 16), __uint_as_float(v & 0xFFFF0000u));
}

__device__ __forceinline__ float ex2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float rcp_approx(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// max(z, lo), a NaN staying a NaN
__device__ __forceinline__ f2 at_least(f2 z, float lo) {
  f2 y;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(y.x) : "f"(z.x), "f"(lo));
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(y.y) : "f"(z.y), "f"(lo));
  return y;
}

// z * sigmoid(u), with t = -u log2 e <= 63.5 or NaN.  The minimum drops a NaN,
// so that one value's never reaches the other; its own z brings it back.
__device__ __forceinline__ f2 mul_sigmoid(f2 z, f2 t) {
  const f2 d = add2(pk(1.0f, 1.0f),
                    pk(ex2_approx(fminf(t.x, 63.5f)), ex2_approx(fminf(t.y, 63.5f))));
  const float r = rcp_approx(d.x * d.y);
  return mul2(z, mul2(pk(d.y, d.x), pk(r, r)));
}

__device__ __forceinline__ f2 act_silu(f2 z) {
  z = at_least(z, -44.0f);
  return mul_sigmoid(z, mul2(z, pk(-1.4426950408889634f, -1.4426950408889634f)));
}

__device__ __forceinline__ f2 act_gelu_tanh(f2 z) {
  // -2 sqrt(2/pi) log2 e (z + 0.044715 z^3)
  constexpr float a = -2.3022082f, b = -0.10294324f;
  z = at_least(z, -7.6f);
  const f2 t = mul2(z, z);
  return mul_sigmoid(z, mul2(z, fma2(t, pk(b, b), pk(a, a))));
}

__device__ __forceinline__ f2 act_gelu(f2 z) {
  z = at_least(z, -13.5f);
  const f2 t0 = mul2(z, z);
  const f2 t = pk(fminf(t0.x, 30.25f), fminf(t0.y, 30.25f));
  f2 q = pk(9.91229884630962e-13f, 9.91229884630962e-13f);
  q = fma2(q, t, pk(-1.5642973028029417e-10f, -1.5642973028029417e-10f));
  q = fma2(q, t, pk(1.0629670477158015e-08f, 1.0629670477158015e-08f));
  q = fma2(q, t, pk(-4.0455273619954824e-07f, -4.0455273619954824e-07f));
  q = fma2(q, t, pk(9.244396096619312e-06f, 9.244396096619312e-06f));
  q = fma2(q, t, pk(-0.00011615729454206303f, -0.00011615729454206303f));
  q = fma2(q, t, pk(-5.883523772354238e-05f, -5.883523772354238e-05f));
  q = fma2(q, t, pk(0.07267936319112778f, 0.07267936319112778f));
  q = fma2(q, t, pk(1.5957502126693726f, 1.5957502126693726f));
  const f2 u = mul2(z, q);
  return mul_sigmoid(z, mul2(u, pk(-1.4426950408889634f, -1.4426950408889634f)));
}

__device__ __forceinline__ f2 act_relu(f2 z) {
  return pk(z.x < 0.0f ? 0.0f : z.x, z.y < 0.0f ? 0.0f : z.y);
}

template <int ACT>
__device__ __forceinline__ f2 act_one(f2 z) {
  if constexpr (ACT == kActRelu) return act_relu(z);
  if constexpr (ACT == kActSilu) return act_silu(z);
  if constexpr (ACT == kActGelu) return act_gelu(z);
  if constexpr (ACT == kActGeluTanh) return act_gelu_tanh(z);
  return z;
}

// f(integral constant of the activation) for `act`, uniform over the launch
template <class F>
__device__ __forceinline__ void with_act(int act, F f) {
  switch (act) {
    case kActRelu: f(std::integral_constant<int, kActRelu>()); break;
    case kActSilu: f(std::integral_constant<int, kActSilu>()); break;
    case kActGelu: f(std::integral_constant<int, kActGelu>()); break;
    case kActGeluTanh: f(std::integral_constant<int, kActGeluTanh>()); break;
    default: f(std::integral_constant<int, kActNone>());
  }
}

// n pairs in place
template <int N>
__device__ __forceinline__ void act_chunk(int act, f2 (&z)[N]) {
  with_act(act, [&](auto a) {
#pragma unroll
    for (int i = 0; i < N; ++i) z[i] = act_one<decltype(a)::value>(z[i]);
  });
}

}  // namespace hq
