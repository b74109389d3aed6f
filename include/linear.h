/*
 * linear.h -- C ABI of the products of few rows with 4-bit weights: the projections around the
 * mixers and the vocabulary head, in the MoE layer's weight format (part of the same library as
 * moe.h).
 *
 * "Optimizing on-device inference for Apple Silicon", section "Decode > Optimize the one-row weight
 * path": a token's products read every weight once, as 4-bit codes with one scale and one bias for
 * each group of 64, and what bounds them is those bytes.
 *
 *     out[t][n] = sum_k x[t][k] (scale[n][k/64] code[n][k] + bias[n][k/64])
 *
 * x is bfloat16 or float16, or the int8 codes and scales that moe_rms_norm gives, in which case
 * sums of products are exact integers within a group of 64.  Codes enter the matrix units as they are (x is
 * not rounded, nor is a dequantised weight); sums are binary32; the result is rounded once.  A group's
 * sum is formed of x (16 + code), which numbers of x up to 2^117 cannot overflow (bfloat16 has larger ones).
 *
 * Conventions are those of attn.h.
 */
#ifndef MOE_LINEAR_MI355X_H
#define MOE_LINEAR_MI355X_H

#include "attn.h"

#ifdef __cplusplus
extern "C" {
#endif

/* (host struct of device pointers) Weights [n][k], in the tiles of moe.h: codes as moe_pack_codes and
 * scale and bias as moe_pack_qparams lay them out, for n rounded up to a multiple of 16 rows and k
 * rounded up to a multiple of 128.  What stands behind row n - 1 is read and has no influence; the
 * scale and bias of a group behind k - 1 must be finite. */
typedef struct {
  const uint32_t *codes;       /* 16-byte aligned */
  const void *scale, *bias;    /* 16-byte aligned */
  int32_t n;                   /* 1 .. 2^24 */
  int32_t k;                   /* a multiple of 64, 64 .. 2^17 */
  moe_dtype qparam_dtype;      /* MOE_FP16 or MOE_BF16 */
} moe_linear_weights;

/* T rows.  Meant for up to some 64 (every 64 read the weights once more).
 *   T          0 .. 2^20 (0: nothing is enqueued); T * n <= 2^40
 *   x          [T][k], rows x_stride elements apart: MOE_BF16 or MOE_FP16, or MOE_INT8 (-127 .. 127; -128
 *              is taken as it is); 16-byte aligned, x_stride * element size a multiple of 16
 *   x_scale    MOE_INT8: float32 [T][k / x_group, or 1], 4-byte aligned; otherwise NULL
 *   x_group    MOE_INT8: 0 (one scale a row), 64 or 128 (dividing k); otherwise 0
 *   out        [T][n] of out_dtype (MOE_BF16, MOE_FP16 or MOE_FP32), rows out_stride elements apart,
 *              aligned to its elements
 * What is written may overlap nothing that is read (MOE_ERR_ALIAS; weights included).
 * MOE_ERR_TOKENS, MOE_ERR_SHAPE, MOE_ERR_DTYPE, MOE_ERR_NULL, MOE_ERR_ALIGN, MOE_ERR_ALIAS,
 * MOE_ERR_DEVICE, MOE_ERR_HIP.  Results are bitwise repeatable.
 * A row of x that holds an infinity or NaN has no finite results; other rows are not touched by it. */
moe_status moe_linear(const moe_linear_weights *w, int64_t T, const void *x, int64_t x_stride, moe_dtype x_dtype,
                      const float *x_scale, int32_t x_group, void *out, int64_t out_stride, moe_dtype out_dtype,
                      hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif
