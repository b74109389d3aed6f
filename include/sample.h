/*
 * sample.h -- C ABI of the choice of tokens from logits, with the random numbers given (part of the
 * same library as moe.h).
 *
 * Per row of V logits l, with weights w_i = exp((l_i - max l) / temperature):
 *   1. tokens of -infinity and NaN are out;
 *   2. top_k > 0 keeps the top_k largest logits (of equal ones, the lowest indices);
 *   3. top_p < 1 keeps, of these in descending order (of equal ones, the lowest index first), the
 *      fewest whose weights sum to at least top_p of their total, and at least one;
 *   4. min_p > 0 keeps those with w_i >= min_p (above 1 it counts as 1);
 *   5. the token is the first i, by index, at which the sum of the kept weights exceeds u times their
 *      total; its probability is its weight over that total.
 * A temperature of 0 (or below, or NaN) takes the largest logit, of equal ones the lowest index, with
 * probability 1.  Numbers that are NaN switch their step off (u: 0); u is cut to [0, 1).  A logit of
 * +infinity counts as the largest float32.  A row without any token gives -1, with probability 0.
 *
 * Weights are held in 64-bit fixed point, with 62 - ceil(log2 V) bits (at most 51) behind that of the
 * largest, or to that precision, so that sums do not depend on their order and results are
 * repeatable.
 *
 * Conventions are those of attn.h.
 */
#ifndef MOE_SAMPLE_MI355X_H
#define MOE_SAMPLE_MI355X_H

#include "moe.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Bytes of workspace for R rows of V logits.  It holds nothing between calls; calls that may run at
 * the same time need one each. */
moe_status moe_sample_workspace(int64_t R, int32_t V, size_t *bytes);

/* R rows (0 .. 65535; 0: nothing is enqueued) of V (1 .. 2^20) logits.
 *   logits       [R][V], rows row_stride elements apart, MOE_FP32, MOE_BF16 or MOE_FP16, aligned to its
 *                elements
 *   u            float32 [R]
 *   temperature, top_p, min_p   float32 [R] or NULL: 1, 1, 0
 *   top_k        int32 [R] or NULL: 0 (0 or below: all tokens)
 *   token        int32 [R]
 *   prob         float32 [R] or NULL
 *   workspace    256-byte aligned
 * Arrays of 4-byte elements are 4-byte aligned.  What is written may overlap nothing else
 * (MOE_ERR_ALIAS).  MOE_ERR_TOKENS (R), MOE_ERR_SHAPE, MOE_ERR_DTYPE, MOE_ERR_NULL, MOE_ERR_ALIGN,
 * MOE_ERR_WORKSPACE, MOE_ERR_ALIAS, MOE_ERR_DEVICE, MOE_ERR_HIP. */
moe_status moe_sample(int64_t R, int32_t V, const void *logits, int64_t row_stride, moe_dtype dtype, const float *u,
                      const float *temperature, const int32_t *top_k, const float *top_p, const float *min_p,
                      int32_t *token, float *prob, void *workspace, size_t workspace_bytes, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif
