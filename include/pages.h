/*
 * pages.h -- C ABI of the paged cache's bookkeeping (part of the same library as moe.h): which
 * pages each sequence holds, kept on the device and changed by kernels, so that a server's step
 * (grow, append, attend) needs no host round trip and can be captured in a graph.  The tables
 * and lengths are the ones that moe_batch of attn.h names.
 *
 * Conventions are those of moe.h: device pointers unless marked (host), caller-owned memory,
 * work enqueued on `stream` without host synchronisation, status codes from moe_status,
 * nothing enqueued on any status but MOE_ERR_HIP.
 *
 * A pool.  Sequence s has len[s] tokens in the pages table[s][0 .. ceil(len[s]/page_size)-1];
 * entries behind those mean nothing.  refs[p] counts the sequences that hold page p; p is free
 * where refs[p] <= 0.  A pool starts as len and refs all zero.
 *
 * Calls.  Each reads the pool `in` and writes the pool `out`, whole: `out` may be `in` (the same
 * three pointers), or share nothing with it -- then `in` is unchanged, and attention that still
 * runs over it stays right until its freed pages are taken.  All sizes of the two must be
 * equal.  Fresh pages are the free ones of lowest number, in the order of the requests, so
 * results depend on the inputs alone.
 *
 * Errors that only the device can see (a request that names a sequence outside the pool, or one
 * twice where it may not; too few free pages; a length behind the table; table entries outside
 * the pool) make the whole call a copy of `in` to `out`, touch no cache, and set *error (sticky,
 * int32 on the device, the first error stays) to the moe_status code named at the call; read it
 * with moe_pages_check.
 */
#ifndef MOE_PAGES_MI355X_H
#define MOE_PAGES_MI355X_H

#include "moe.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct {               /* (host struct of device pointers), 4-byte aligned */
  int32_t *table;              /* [n_seqs][table_cols] */
  int32_t *len;                /* [n_seqs] tokens */
  int32_t *refs;               /* [n_pages] */
  int32_t n_seqs;              /* 1 .. 65535 */
  int32_t table_cols;          /* >= 1; table_cols * page_size <= 2^30; n_seqs * table_cols < 2^31 */
  int32_t n_pages;             /* 1 .. 2^26 */
  int32_t page_size;           /* tokens: a power of two, 1 .. 65536 */
} moe_pages;

/* The memory of the pages: n_planes planes (keys and values of each layer), in each of which a
 * page is page_bytes contiguous bytes at page * page_stride.  All are multiples of 16 bytes,
 * and base is 16-byte aligned. */
typedef struct {
  void *base;
  int64_t plane_stride;        /* bytes, >= (n_pages - 1) * page_stride + page_bytes (any for one
                                  plane), or the planes of a page lie inside page_stride */
  int64_t page_stride;         /* bytes */
  int64_t page_bytes;          /* 16 .. 2^30 */
  int32_t n_planes;            /* 1 .. 65535 */
} moe_page_memory;

/* Bytes of workspace (256-byte aligned) that every call below needs for a pool of these sizes and
 * n requests.  It holds nothing between calls. */
moe_status moe_pages_workspace(const moe_pages *pages, int32_t n, size_t *bytes);

/* n sequences grow by tokens[i] >= 0 tokens each (0 .. 2^30): pages are added where the last one
 * has no room.  seqs: distinct.  MOE_ERR_SHAPE (a sequence outside the pool or twice, a negative
 * or too long growth), MOE_ERR_ALLOC (too few free pages).
 * A page that other sequences share is appended to only if it is full: moe_pages_fork copies
 * a last page that is not. */
moe_status moe_pages_grow(const moe_pages *in, const moe_pages *out, int32_t n, const int32_t *seqs,
                          const int32_t *tokens, int32_t *error, void *workspace, size_t workspace_bytes,
                          hipStream_t stream);

/* dst[i] becomes a copy of src[i]: full pages are shared (their refs grow), and a last page that
 * is not full is copied in every plane to a fresh page.  dst: distinct, empty (len 0), no src
 * among them; a src may occur any number of times.  MOE_ERR_SHAPE, MOE_ERR_ALLOC. */
moe_status moe_pages_fork(const moe_pages *in, const moe_pages *out, const moe_page_memory *mem, int32_t n,
                          const int32_t *src, const int32_t *dst, int32_t *error, void *workspace,
                          size_t workspace_bytes, hipStream_t stream);

/* n sequences end: their length becomes 0 and the refs of their pages shrink.  seqs: distinct.
 * MOE_ERR_SHAPE. */
moe_status moe_pages_free(const moe_pages *in, const moe_pages *out, int32_t n, const int32_t *seqs,
                          int32_t *error, void *workspace, size_t workspace_bytes, hipStream_t stream);

/* The u pages in use move to the numbers 0 .. u-1: those at u and behind it go, in order, to the
 * free numbers below u, in order; tables and refs follow.  Only free pages are written, so a
 * pool `in` other than `out` stays readable.  MOE_ERR_SHAPE where a table entry of a sequence is
 * outside the pool. */
moe_status moe_pages_compact(const moe_pages *in, const moe_pages *out, const moe_page_memory *mem,
                             int32_t *error, void *workspace, size_t workspace_bytes, hipStream_t stream);

/* Page src[i] is copied to page dst[i] in every plane, i < n (dst: distinct, no src among them;
 * otherwise those pages' contents are undefined).  A pair with a number outside [0, n_pages) is
 * skipped.  n: 0 .. 2^20. */
moe_status moe_pages_copy(const moe_page_memory *mem, int32_t n_pages, int32_t n, const int32_t *src,
                          const int32_t *dst, hipStream_t stream);

/* MOE_OK, or the first error that a call left in *error since it was cleared (a 4-byte zero);
 * waits for the stream.  MOE_ERR_HIP if the copy failed. */
moe_status moe_pages_check(const int32_t *error, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif
