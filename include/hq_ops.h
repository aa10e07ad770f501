/* hq_ops.h -- C ABI of the operators beside the quantized linear layer: the
 * matrix products with an activation, a gate and a residual in their epilogue
 * (on the layer's codes and on 16-bit operands), and the group norm with an
 * activation over channels-last tensors.  With hq.h they make up the blocks
 * that the layer sits in:
 *
 *   transformer MLP   hq_quantize_act -> hq_linear_ep (fc1, GELU)
 *                     -> hq_quantize_act -> hq_linear_ep (fc2, gate, residual),
 *                     the gate a row per sample from hq_dense;
 *   1x1 convolution   hq_group_norm (SiLU) -> hq_quantize_act
 *                     -> hq_linear_ep (residual), pixels as tokens (NHWC).
 *
 * Conventions are hq.h's: device pointers owned by the caller, row-major
 * matrices, bf16 as uint16_t bit patterns, calls asynchronous on `stream`,
 * errors returned and checked before any launch, no allocation, no
 * synchronization.  A call keeps no state between calls, may be captured in a
 * graph, and may run beside other calls on other streams as long as they share
 * no buffer that one of them writes (workspaces included). */
#ifndef HQ_OPS_H_
#define HQ_OPS_H_

#include <stddef.h>
#include <stdint.h>

#include "hq.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Activations, applied in fp32 to the value z that enters them:
 *   HQ_ACT_NONE       z
 *   HQ_ACT_RELU       max(z, 0)
 *   HQ_ACT_SILU       z / (1 + e^-z)
 *   HQ_ACT_GELU       z Phi(z) = z (1 + erf(z / sqrt 2)) / 2
 *   HQ_ACT_GELU_TANH  z (1 + tanh(sqrt(2/pi) (z + 0.044715 z^3))) / 2
 * A NaN stays a NaN.  In fp32, before the stored rounding, silu and gelu_tanh are
 * z sigmoid(u), with u = z and u = 2 sqrt(2/pi) (z + 0.044715 z^3), and are off by
 * at most 2^-20 (1 + |u| / 4) of their value plus 7e-18: the exponential's and the
 * reciprocal's own error, and the rounding of the exponent, which grows with u
 * (|u| <= 44; the value itself is within 7e-18 of 0 from u = -43.3 down).  HQ_ACT_GELU is off by at most
 * 2^-16 of its value plus 1.1e-7 (the fit of its exponent).  Of -infinity they give
 * their limit to that error. */
enum {
  HQ_ACT_NONE = 0,
  HQ_ACT_RELU = 1,
  HQ_ACT_SILU = 2,
  HQ_ACT_GELU = 3,
  HQ_ACT_GELU_TANH = 4
};

/* What a product does with z[t,n], the value it would store without one
 * (host memory, passed by const pointer):
 *
 *   Y[t,n] = bf16_rne( residual[t,n] + gate[t / gate_rows, n] * act(z[t,n]) )
 *
 * in fp32, rounded once.
 *   act        HQ_ACT_*.
 *   residual   bf16 [T,N] (device), or NULL (0).  May be Y itself (the
 *              product is then added in place), but may not overlap it
 *              otherwise.
 *   gate       bf16 [ceil(T / gate_rows), N] (device), or NULL (1): one row
 *              for each gate_rows rows of Y, such as a sample's modulation.
 *   gate_rows  >= 1 with a gate; not read without one. */
typedef struct hq_epilogue {
  int32_t act;
  const uint16_t* residual;
  const uint16_t* gate;
  int64_t gate_rows;
} hq_epilogue;

/* hq_linear_ep -- hq_linear with an epilogue: z is the layer's output before
 * its rounding,
 *   z[t,n] = s_x[t] * w_scale[n] * acc[t,n] + bias_f32[n] + a_mean[t] * colsum[n],
 * or, in the weight-only Hadamard form, the output-side transform's result
 * plus bias.  Every description, code format and argument of hq_linear;
 * `epilogue` may be NULL (the results are then those of hq_linear, bit for bit).
 * N is a multiple of 16, N <= 2^30 and T <= 2^31 - 256. */
hq_status hq_linear_ep(const hq_layer_desc* desc, int64_t T, const int8_t* a_codes,
                       const float* a_scale, const float* a_mean, const int8_t* w_codes,
                       const float* w_scale, const float* colsum, const float* bias_f32,
                       const hq_epilogue* epilogue, uint16_t* Y, int32_t* acc_debug,
                       hq_stream_t stream);

/* A 16-bit linear layer: K input and N output channels, both multiples of 8;
 * K <= 2^20, N <= 2^30. */
typedef struct hq_dense_desc {
  int32_t K, N;
} hq_dense_desc;

/* hq_dense -- a linear layer that stays in 16 bits (a timestep or modulation
 * MLP, a first or last layer), with the same epilogue:
 *   z[t,n] = sum_k X[t,k] W[n,k] + bias[n]      (fp32 sums)
 * Inputs:  X bf16 [T,K], W bf16 [N,K] (the nn.Linear orientation), bias bf16
 *          [N] or NULL; `epilogue` may be NULL (Y = bf16(z)).
 * Output:  Y bf16 [T,N]; it overlaps no input but the residual it may equal.
 * T >= 0 (T = 0 is a no-op), T <= 2^31 - 256.  All pointers 16-byte aligned.
 * Results are deterministic: every sum over K is taken in an order that
 * depends on the sizes, on whether there is an activation (the kernel's choice
 * goes by it) and on the device's SM count alone. */
hq_status hq_dense(const hq_dense_desc* desc, const uint16_t* X, int64_t T, const uint16_t* W,
                   const uint16_t* bias, const hq_epilogue* epilogue, uint16_t* Y,
                   hq_stream_t stream);

/* Group norm over channels-last tensors: C channels in `groups` groups of
 * C / groups consecutive channels (groups divides C; C <= 8192; any group
 * size), eps >= 0, and an activation. */
typedef struct hq_group_norm_desc {
  int32_t C, groups;
  int32_t act; /* HQ_ACT_* */
  float eps;
} hq_group_norm_desc;

/* Bytes of device workspace hq_group_norm needs for B images of S pixels on the
 * current device: 0 where it needs none (small tensors), where there is nothing
 * to do, and for a description that the call refuses. */
size_t hq_group_norm_workspace_bytes(const hq_group_norm_desc* desc, int64_t B, int64_t S);

/* hq_group_norm -- over every image b and group g, with the mean and the
 * (population) variance of its S * C / groups values:
 *   Y[b,s,c] = bf16_rne( act( (X[b,s,c] - mean) / sqrt(var + eps) * gamma[c] + beta[c] ) )
 * Inputs:  X bf16 [B,S,C]; gamma, beta bf16 [C] or NULL (1 and 0).
 * Output:  Y bf16 [B,S,C]; may be X itself, may not overlap it otherwise.
 * workspace: device, 16-byte aligned, >= hq_group_norm_workspace_bytes()
 *   bytes (NULL where that is 0); contents need not be initialised.
 * Statistics are held in fp32 as means and sums of squared deviations around a
 * value of the group (never a difference of large sums), in an order that
 * depends on the sizes and the device's SM count alone.  A NaN or an infinity
 * makes its image's group NaN and touches no other, and so do finite values
 * whose squared deviations add up past fp32's range (3.4e38; deviations below
 * 1e-22 count as none).  B = 0 or S = 0 is a no-op.
 * B, S < 2^31.  X, Y, gamma and beta 16-byte aligned. */
hq_status hq_group_norm(const hq_group_norm_desc* desc, const uint16_t* X, int64_t B, int64_t S,
                        const uint16_t* gamma, const uint16_t* beta, uint16_t* Y, void* workspace,
                        size_t workspace_bytes, hq_stream_t stream);

/* ---------------------------------------------------------------------------
 * Test hooks: which kernel a product with an epilogue runs.
 *   HQ_PRODUCT_ROWS    one pass over the weights from registers, T <= 8;
 *                      width: the token count it is built for (1, 2, 4, 8),
 *                      split: warps that share a row's K (1, 2, 4);
 *   HQ_PRODUCT_SPLIT   K split over a cluster; width: tokens per tile (16, 32,
 *                      64, 128), split: CTAs per cluster (1, 2, 4, 8);
 *   HQ_PRODUCT_TILES   one CTA per 128 x width tile (64, 128, 192, 256);
 *   HQ_PRODUCT_PAIR    two CTAs per 256 x width tile (128, 192, 256);
 *   HQ_PRODUCT_LINEAR  hq_linear's own kernel (a plain epilogue on codes);
 *                      width its tile's, split 2 for the CTA pair.
 * Where width or split are not named they are 1 in what a query returns, and
 * not read of what is set. */
enum {
  HQ_PRODUCT_AUTO = 0,
  HQ_PRODUCT_ROWS = 1,
  HQ_PRODUCT_SPLIT = 2,
  HQ_PRODUCT_TILES = 3,
  HQ_PRODUCT_PAIR = 4,
  HQ_PRODUCT_LINEAR = 5
};
typedef struct hq_product_plan {
  int32_t kernel, width, split;
} hq_product_plan;

/* Host only (no device call): the plan of hq_dense and hq_linear_ep for T
 * tokens on a device with `sms` SMs that holds `pair_clusters` CTA-pair
 * clusters.  act: the epilogue's; plain != 0: there is none (and no raw
 * accumulators are asked for).  HQ_ERR_UNSUPPORTED where a plan is set that
 * cannot run the product. */
hq_status hq_debug_dense_plan(const hq_dense_desc* desc, int64_t T, int act, int sms,
                              int pair_clusters, hq_product_plan* plan);
hq_status hq_debug_linear_ep_plan(const hq_layer_desc* desc, int64_t T, int plain, int act, int sms,
                                  int pair_clusters, hq_product_plan* plan);

/* Host state, applies to calls issued after it: the plan that hq_dense and
 * hq_linear_ep take instead of choosing one (NULL or HQ_PRODUCT_AUTO: the
 * default).  They return HQ_ERR_UNSUPPORTED for a product that it cannot run:
 * ROWS past 8 tokens, SPLIT with fewer 128-byte K blocks than CTAs, PAIR for
 * packed codes or the weight-only form, ROWS and SPLIT for the weight-only form
 * or with raw accumulators, SPLIT and 256-column tiles for packed codes. */
hq_status hq_debug_set_product_plan(const hq_product_plan* plan);

#ifdef __cplusplus
}
#endif

#endif /* HQ_OPS_H_ */
