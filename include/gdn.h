/*
 * gdn.h -- C ABI of the Gated DeltaNet prefill scan and decode step (part of the same library
 * as moe.h).
 *
 * "Optimizing on-device inference for Apple Silicon", section "Prefill > Keep recurrent
 * state on chip": during prefill a Gated DeltaNet layer scans the prompt in order and
 * carries a recurrent state matrix; the state and its gate are 32-bit floats, query and
 * key activations bfloat16.  The pages print no update formula; the one implemented is
 * the gated delta rule (Yang, Kautz and Hatamizadeh, "Gated Delta Networks", ICLR 2025),
 * per value head h and token t:
 *
 *     S_t = alpha_t S_{t-1} (I - beta_t k_t k_t^T) + beta_t v_t k_t^T
 *     o_t = S_t q_t
 *
 * S is d_v x d_k with one row per value channel; value head h reads key head
 * h / (n_vheads / n_kheads).  The state stays in registers for the whole scan (one
 * 16-lane group per row) and is written back once at the end.
 *
 * Conventions are those of moe.h: device pointers, caller-owned memory, work enqueued
 * on `stream` without host synchronisation, status codes from moe_status.
 */
#ifndef MOE_GDN_MI355X_H
#define MOE_GDN_MI355X_H

#include "moe.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Scan T tokens of one layer, starting from the state in `state` and leaving the state
 * after token T-1 there (so a long prompt can be scanned in chunks, the state carried
 * from one call to the next; section "Prefill > Bound temporary memory with prompt
 * chunking").
 *   T          tokens, >= 0 (0: nothing is enqueued, the state is unchanged)
 *   n_kheads   key/query heads >= 1; n_vheads value heads, a multiple of n_kheads, <= 4096
 *   d_k, d_v   head widths; both must be 128
 *   q, k       bf16 [T][n_kheads][128], 16-byte aligned
 *   v          bf16 [T][n_vheads][128], 16-byte aligned
 *   alpha      float32 [T][n_vheads]: the decay gate (in [0, 1] for the intended use;
 *              0 clears the state before the token's write), 4-byte aligned
 *   beta       float32 [T][n_vheads]: the write strength, 4-byte aligned
 *   state      float32 [n_vheads][128][128] (row j = value channel j), read and
 *              written in place, 16-byte aligned
 *   out        bf16 [T][n_vheads][128], o_t rounded to nearest even, 2-byte aligned
 * out and state may overlap neither an input nor each other (MOE_ERR_ALIAS).
 * Returns MOE_ERR_TOKENS (T < 0), MOE_ERR_SHAPE, MOE_ERR_NULL, MOE_ERR_ALIGN,
 * MOE_ERR_DEVICE (current device not gfx950) or MOE_ERR_HIP, before enqueueing anything
 * except for MOE_ERR_HIP. */
moe_status moe_gdn_scan(int32_t T, int32_t n_kheads, int32_t n_vheads, int32_t d_k, int32_t d_v,
                        const void *q, const void *k, const void *v, const float *alpha,
                        const float *beta, float *state, void *out, hipStream_t stream);

/* One token each of R rows, for serving: row r brings one token of the sequence whose state is
 * slot[r] of a pool of states, which is read and written in place (the update of
 * moe_gdn_scan).  Rows of one slot are applied in row order, so a few tokens of one sequence
 * (a draft to verify) may follow each other as rows; different slots are independent.
 *   R          rows, >= 0 (0: nothing is enqueued); R * n_vheads <= 2^20 (MOE_ERR_TOKENS)
 *   n_kheads   key/query heads >= 1; n_vheads value heads, a multiple of n_kheads, <= 4096
 *   d_k, d_v   head widths; both must be 128
 *   q, k       bf16 [R][n_kheads][128], 16-byte aligned
 *   v          bf16 [R][n_vheads][128], 16-byte aligned
 *   alpha      float32 [R][n_vheads], beta float32 [R][n_vheads], 4-byte aligned
 *   state      float32 [n_slots][n_vheads][128][128] (row j = value channel j), 16-byte aligned
 *   slot       int32 [R], 4-byte aligned: a row whose slot lies outside [0, n_slots) is
 *              padding: it touches no state, and its output is zeros
 *   out        bf16 [R][n_vheads][128], o_t rounded to nearest even, 2-byte aligned
 * A decay of 0 takes the slot's old state as zeros whatever it holds, so a slot starts a new
 * sequence without being cleared.  Every row looks through the slots for its like, which is meant
 * for up to some thousand rows.
 * out and state may overlap neither an input nor each other (MOE_ERR_ALIAS).  Status codes as
 * moe_gdn_scan (MOE_ERR_SHAPE also for n_slots < 1).  May be captured in a graph: slot is
 * read when the kernel runs. */
moe_status moe_gdn_step(int32_t R, int32_t n_kheads, int32_t n_vheads, int32_t d_k, int32_t d_v,
                        const void *q, const void *k, const void *v, const float *alpha,
                        const float *beta, float *state, int32_t n_slots, const int32_t *slot, void *out,
                        hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif
