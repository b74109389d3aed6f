/*
 * attn.h -- C ABI of the attention mixer's serving operators (part of the same library as
 * moe.h): query/key preparation with the append to a paged cache, and attention of new
 * tokens over that cache.
 *
 * "Optimizing on-device inference for Apple Silicon": the model alternates Gated DeltaNet
 * layers (gdn.h) with full-attention layers of 16 query and 2 key/value heads of width 256;
 * prompts run in chunks between which the key/value cache is kept (section "Prefill >
 * Bound temporary memory with prompt chunking"), and the query heads that share a key/value
 * head share its loads (section "Decode > Read the attention cache efficiently").
 *
 * Conventions are those of moe.h: device pointers unless marked (host), caller-owned
 * memory, work enqueued on `stream` without host synchronisation (so every call may be
 * captured in a graph), status codes from moe_status, nothing enqueued on any status but
 * MOE_ERR_HIP.  Strides are in elements.
 *
 * The cache.  Keys and values live in pages of page_size tokens; element (page, token,
 * head, i) is at page * page_stride + token * token_stride + head * head_stride + i of the
 * k and of the v array.  A sequence's token at position p is token p % page_size of page
 * table[row][p / page_size].
 *
 * A batch.  n_seqs sequences bring q_start[n_seqs] new tokens, stacked: sequence b's are
 * tokens q_start[b] .. q_start[b+1]-1 (n_b of them; none is fine) of the token-indexed
 * arrays, which have T >= q_start[n_seqs] tokens; tokens behind the last sequence are
 * padding, and nothing is written for them.  Sequence b uses table row r = row[b] (b where
 * row is NULL); kv_len[r] is its length INCLUDING the new tokens, so new token i sits at
 * position kv_len[r] - n_b + i.
 *
 * The device arrays are not known to the host, so the kernels check them: a row outside
 * [0, n_rows) counts as a sequence of length 0, a length above table_cols * page_size is
 * cut there for what is read and written, and a page number outside [0, n_pages) is never
 * read or written (its keys count as absent, its tokens are not stored).  q_start has to
 * ascend from 0; where it does not, outputs are undefined but no access leaves the arrays.
 */
#ifndef MOE_ATTN_MI355X_H
#define MOE_ATTN_MI355X_H

#include "moe.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct {               /* (host struct of device pointers) [T][heads][head_dim] */
  const void *p;               /* 16-byte aligned */
  int64_t token_stride;        /* multiples of 8, >= 0 */
  int64_t head_stride;
} moe_heads;

typedef struct {               /* (host struct of device pointers) */
  void *k, *v;                 /* 16-byte aligned; the same strides */
  int64_t page_stride;         /* multiples of 8; no two elements may share a place; one */
  int64_t token_stride;        /* page's elements span less than 2^30 */
  int64_t head_stride;
  int32_t n_pages;             /* >= 1 */
  int32_t page_size;           /* a power of two, 16 .. 65536 */
  int32_t n_kv_heads;          /* 1 .. 1024 */
  int32_t head_dim;            /* 64, 128 or 256 */
  moe_dtype dtype;             /* MOE_BF16 or MOE_FP16: of the cache and of q, k, v, out */
} moe_paged_kv;

typedef struct {               /* (host struct of device pointers), 4-byte aligned */
  const int32_t *q_start;      /* [n_seqs + 1] */
  const int32_t *kv_len;       /* [n_rows] */
  const int32_t *table;        /* [n_rows][table_cols] */
  const int32_t *row;          /* [n_seqs] or NULL */
  int32_t n_seqs;              /* 1 .. 65535 */
  int32_t n_rows;              /* >= 1; >= n_seqs where row is NULL */
  int32_t table_cols;          /* >= 1; table_cols * page_size <= 2^30 */
} moe_batch;

/* Rotary frequencies (host; no device work).  out[i], i < rot_dim / 2, gets the angle per
 * position of pair i: base^(-2i/rot_dim), stretched for contexts longer than trained ones:
 *   MOE_ROPE_NONE    as it is
 *   MOE_ROPE_LINEAR  divided by factor (positions interpolated)
 *   MOE_ROPE_NTK     of the base base * factor^(rot_dim / (rot_dim - 2))
 *   MOE_ROPE_YARN    by the pair's turns over the trained length, t = trained * f / 2 pi:
 *                    f where t >= 32, f / factor where t <= 1, linear in t between (Peng et
 *                    al., "YaRN: Efficient Context Window Extension of Large Language
 *                    Models", ICLR 2024); *mscale = 0.1 ln(factor) + 1.  Models trained with
 *                    another ramp between the two (linear in the pair's index i, say) need
 *                    frequencies of their own: moe_rope_append takes any
 * *mscale is 1 for the others.  rot_dim: even, 2 .. 256 (NTK: >= 4); base > 1; factor >= 1;
 * trained >= 1 (read for YARN only).  MOE_ERR_NULL, MOE_ERR_SHAPE. */
typedef enum { MOE_ROPE_NONE = 0, MOE_ROPE_LINEAR = 1, MOE_ROPE_NTK = 2, MOE_ROPE_YARN = 3 } moe_rope_scaling;
moe_status moe_rope_freqs(int32_t rot_dim, double base, moe_rope_scaling scaling, double factor,
                          int64_t trained, double *out, float *mscale);

/* Query/key preparation of T new tokens and their append to the cache, in one launch.
 * The first rot_dim elements of each query and key head are rotated pair by pair by the
 * angle pos * inv_freq[i],
 *     a' = mscale (a cos - b sin),   b' = mscale (a sin + b cos),
 * pairs (i, i + rot_dim/2), or (2i, 2i+1) with MOE_ROPE_INTERLEAVED; the other elements
 * pass unchanged.  Angles are reduced in binary64, the rotation is binary32, rounded once.
 * Rotated queries go to q_out, rotated keys and unchanged values to their cache places.
 *   pos       int32 [T], or NULL: the token's position in its sequence
 *   inv_freq  binary64 [rot_dim / 2], 8-byte aligned (NULL where rot_dim is 0)
 *   rot_dim   even, 0 .. head_dim
 *   n_heads   query heads, 0 .. 4096 (0: q and q_out are not read)
 *   k, v      [T][n_kv_heads][head_dim]; both p NULL: nothing is appended, and the cache's
 *             k and v may be NULL too
 *   q_out     may be q itself (same p and strides); otherwise what is written may overlap
 *             nothing that is read
 * A token whose position is negative or lies behind the table is not appended.  Two tokens
 * of one cache place (sequences that share a page which is not full) race: moe_pages_fork
 * never leaves such a page.  T: 0 .. 2^20 (MOE_ERR_TOKENS). */
#define MOE_ROPE_INTERLEAVED 1u
moe_status moe_rope_append(const moe_paged_kv *kv, const moe_batch *batch, int64_t T, const moe_heads *q,
                           const moe_heads *q_out, int32_t n_heads, const moe_heads *k, const moe_heads *v,
                           const int32_t *pos, const double *inv_freq, int32_t rot_dim, float mscale,
                           uint32_t flags, hipStream_t stream);

/* Attention of the batch's new tokens over the cache (which already holds their keys and
 * values): per new token i of sequence b, at position p, and query head h, with key/value
 * head h / (n_heads / n_kv_heads),
 *     out = sum_j softmax_j(scale * q . k_j) v_j
 * over the positions j < kv_len that it sees: j <= p (all of them with MOE_ATTN_FULL), and
 * j > p - window where window > 0.  A token that sees nothing, or whose scores are all
 * -infinity, gets zeros, and a log-sum-exp of -infinity.  Positions it does not see have no
 * influence, whatever their cache places hold (NaN among it).
 *   max_q, max_kv  (host) upper bounds of n_b and kv_len that the launch is shaped by.
 *                  Smaller numbers than the true ones cost time, not results.
 *   q, out         [T][n_heads][head_dim]; n_heads a multiple of n_kv_heads, <= 4096
 *   lse            float32 [T][n_heads] or NULL: natural log of the sum of exp(scale q . k)
 *   scale          finite, also times log2(e)
 *   window         >= 0; 0 with MOE_ATTN_FULL
 *   workspace      256-byte aligned, at least the bytes that moe_paged_attn_workspace gives
 *                  for the same sizes; may be NULL where that is 0.  It holds nothing
 *                  between calls; calls that may run at the same time need one each.
 * out and lse may overlap nothing that is read, the workspace, or each other
 * (MOE_ERR_ALIAS).  Scores, softmax statistics and sums are binary32; the weights of the
 * value sum are rounded to dtype (they enter the matrix units in it), those of fp16 below
 * 2^-25 of the row's largest one by at most 2^-36 of that.  For one shape of launch, results
 * are bitwise repeatable.  T: 0 .. 2^20, T * n_heads <= 2^29, n_seqs * n_kv_heads <= 2^22
 * (MOE_ERR_TOKENS). */
#define MOE_ATTN_FULL 1u
moe_status moe_paged_attn_workspace(const moe_paged_kv *kv, int64_t T, int32_t n_seqs, int64_t max_q,
                                    int64_t max_kv, int32_t n_heads, int32_t window, size_t *bytes);
moe_status moe_paged_attn(const moe_paged_kv *kv, const moe_batch *batch, int64_t T, int64_t max_q,
                          int64_t max_kv, const moe_heads *q, int32_t n_heads, const moe_heads *out,
                          float *lse, float scale, int32_t window, uint32_t flags, void *workspace,
                          size_t workspace_bytes, hipStream_t stream);

/* Groups of a batch's sequences that share a prefix, as moe_pages_fork leaves them: group g is the
 * sequences group_start[g] .. group_start[g+1]-1 (consecutive; one alone is fine), and the first
 * prefix_len[g] positions (0 is fine) of all of them hold the same keys and values.  group_start has to
 * ascend from 0 to n_seqs; where it does not, outputs are undefined but no access leaves the
 * arrays. */
typedef struct {               /* (host struct of device pointers), 4-byte aligned */
  const int32_t *group_start;  /* [n_groups + 1] */
  const int32_t *prefix_len;   /* [n_groups] */
  int32_t n_groups;            /* 1 .. n_seqs */
} moe_prefix_groups;

/* moe_paged_attn for such a batch: a prefix's keys and values are read once for the tokens of all
 * sequences of its group, through the table row of the group's first sequence (a row outside the
 * table: the prefix is absent), and each sequence's own positions behind it through its row; the two are
 * joined.  Every new token has to stand behind its prefix: it sees the whole of it, wherever it stands, and
 * of the positions from prefix_len on those that moe_paged_attn without a window shows it (of a
 * sequence whose own row lies outside the table: none).
 *   max_q, max_prefix, max_suffix   (host) upper bounds of n_b, of prefix_len and of kv_len - prefix_len
 *                that the launch is shaped by.  Smaller numbers than the true ones cost time, not results.
 * Other arguments and errors as moe_paged_attn; the workspace is never empty.  T * n_heads <= 2^20
 * (MOE_ERR_TOKENS): meant for single tokens and drafts. */
moe_status moe_prefix_attn_workspace(const moe_paged_kv *kv, int64_t T, int32_t n_seqs, int32_t n_groups, int64_t max_q,
                                     int64_t max_prefix, int64_t max_suffix, int32_t n_heads, size_t *bytes);
moe_status moe_prefix_attn(const moe_paged_kv *kv, const moe_batch *batch, const moe_prefix_groups *groups, int64_t T,
                           int64_t max_q, int64_t max_prefix, int64_t max_suffix, const moe_heads *q, int32_t n_heads,
                           const moe_heads *out, float *lse, float scale, uint32_t flags, void *workspace,
                           size_t workspace_bytes, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif
