/*
 * norm.h -- C ABI of the root-mean-square norm that stands before and inside the mixers and the
 * MoE layer, with the residual's addition and an output in 8 bits (part of the same library as
 * moe.h).
 *
 * Per row x of `width` elements, with an optional residual r:
 *     h = x + r                                        (binary32; stored rounded to dtype)
 *     y = h * (mean(h^2) + eps)^(-1/2) * (offset + w)   (from the unrounded h)
 * y is rounded once, to dtype, or to 8 bits with scales: of each `group` elements of a row
 * (whole rows: group 0) s = max|y| / 127 and code = y / s rounded to the nearest integer (ties to
 * even), or s = max|y| / 448 and code = y / s rounded to the nearest e4m3 number (without infinities).
 * A group of zeros (or of nothing that reaches 2^-120) has scale and codes 0; one with an infinity or NaN has
 * scale infinity or NaN and codes 0.  The sum of squares is binary32.
 *
 * linear.h takes int8 with a scale for each row or for each 64 or 128 elements; int8 by 32 and e4m3 are for
 * products outside this library.
 *
 * Conventions are those of attn.h.
 */
#ifndef MOE_NORM_MI355X_H
#define MOE_NORM_MI355X_H

#include "attn.h"

#ifdef __cplusplus
extern "C" {
#endif

/* T tokens of n_heads rows each.
 *   width      1 .. 2^20; n_heads 1 .. 4096; T 0 .. 2^20 (0: nothing is enqueued), T * n_heads <= 2^28
 *   dtype      MOE_BF16 or MOE_FP16: of x, residual, sum, weight
 *   x          [T][n_heads][width]; any strides >= 0, 2-byte aligned (16-byte aligned rows of a multiple
 *              of 8 elements are a little faster)
 *   residual   the same, or NULL: nothing is added
 *   sum        h, or NULL (needs no residual).  May be x or residual itself (same address and
 *              strides).
 *   weight     [width], 2-byte aligned, or NULL: y = h * rsqrt(...) * offset
 *   out_dtype  dtype, MOE_INT8 or MOE_FP8
 *   out        [T][n_heads][width] in out_dtype (strides in its elements).  Of dtype: may be x or
 *              residual itself.
 *   group      8-bit outputs: 0 (whole rows), or 32, 64 or 128 dividing width (x, residual, sum
 *              and weight 16-byte and out 8-byte aligned, strides multiples of 8, MOE_ERR_ALIGN);
 *              otherwise 0
 *   scale      8-bit outputs: float32 [T][n_heads][width / group, or 1]; otherwise NULL
 *   eps        >= 0, finite (0: a row whose squares vanish in binary32 has no number: zeros give NaN); offset finite
 * What is written may otherwise overlap nothing that is read or written (MOE_ERR_ALIAS).
 * MOE_ERR_TOKENS, MOE_ERR_SHAPE, MOE_ERR_DTYPE, MOE_ERR_NULL, MOE_ERR_ALIGN, MOE_ERR_ALIAS,
 * MOE_ERR_DEVICE, MOE_ERR_HIP. */
moe_status moe_rms_norm(int64_t T, int32_t n_heads, int32_t width, moe_dtype dtype, const moe_heads *x,
                        const moe_heads *residual, const moe_heads *sum, const void *weight, float offset, float eps,
                        moe_dtype out_dtype, const moe_heads *out, int32_t group, float *scale, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif
