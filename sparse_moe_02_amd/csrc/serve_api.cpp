// Host side of the C ABI declared in include/attn.h and include/pages.h and of moe_gdn_step
// (include/gdn.h):
// argument checks and launches.  Every check precedes every launch.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "../../include/attn.h"
#include "../../include/gdn.h"
#include "../../include/pages.h"
#include "checks.hpp"
#include "kernels.hpp"

using namespace moe;

namespace {

moe_status check_kv(const moe_paged_kv *kv, bool planes) {
  if (!kv) return MOE_ERR_NULL;
  if (kv->dtype != MOE_BF16 && kv->dtype != MOE_FP16) return MOE_ERR_DTYPE;
  if (kv->head_dim != 64 && kv->head_dim != 128 && kv->head_dim != 256) return MOE_ERR_SHAPE;
  if (kv->n_kv_heads < 1 || kv->n_kv_heads > 1024 || kv->n_pages < 1) return MOE_ERR_SHAPE;
  if (kv->page_size < 16 || kv->page_size > 65536 || (kv->page_size & (kv->page_size - 1))) return MOE_ERR_SHAPE;
  if (!planes) return MOE_OK;
  if (!kv->k || !kv->v) return MOE_ERR_NULL;
  if (!aligned(kv->k, 16) || !aligned(kv->v, 16)) return MOE_ERR_ALIGN;
  if (kv->page_stride < 0 || kv->token_stride < 0 || kv->head_stride < 0) return MOE_ERR_SHAPE;
  if (kv->page_stride % 8 || kv->token_stride % 8 || kv->head_stride % 8) return MOE_ERR_ALIGN;
  const __int128 page = (__int128)(kv->page_size - 1) * kv->token_stride +
                        (__int128)(kv->n_kv_heads - 1) * kv->head_stride + kv->head_dim;
  if (page >= (__int128)1 << 30) return MOE_ERR_SHAPE;
  Dim d[3] = {{kv->page_stride, kv->n_pages}, {kv->token_stride, kv->page_size}, {kv->head_stride, kv->n_kv_heads}};
  return distinct(d, 3, kv->head_dim) ? MOE_OK : MOE_ERR_SHAPE;
}
Span kv_span(const moe_paged_kv &kv, const void *p) {
  return Span{p, (uint64_t)(2 * ((kv.n_pages - 1) * kv.page_stride + (kv.page_size - 1) * kv.token_stride +
                                 (kv.n_kv_heads - 1) * kv.head_stride + kv.head_dim))};
}

// Whether the two planes may share elements.  Planes that interleave page by page (one
// allocation [page][2][...]) are compared within a page.
bool planes_overlap(const moe_paged_kv &kv) {
  if (!overlap(kv_span(kv, kv.k), kv_span(kv, kv.v))) return false;
  const int64_t ps = 2 * kv.page_stride;
  const int64_t w = 2 * ((kv.page_size - 1) * kv.token_stride + (kv.n_kv_heads - 1) * kv.head_stride + kv.head_dim);
  if (ps == 0 || w > ps) return true;
  int64_t d = (int64_t)((uintptr_t)kv.k - (uintptr_t)kv.v) % ps;
  if (d < 0) d += ps;
  return !(d >= w && d + w <= ps);
}

moe_status check_batch(const moe_batch *b, int32_t page_size) {
  if (!b || !b->q_start || !b->kv_len || !b->table) return MOE_ERR_NULL;
  if (b->n_seqs < 1 || b->n_seqs > 65535 || b->n_rows < 1 || (!b->row && b->n_rows < b->n_seqs)) return MOE_ERR_SHAPE;
  if (b->table_cols < 1 || (int64_t)b->table_cols * page_size > int64_t(1) << 30) return MOE_ERR_SHAPE;
  if (!aligned(b->q_start, 4) || !aligned(b->kv_len, 4) || !aligned(b->table, 4) || !aligned(b->row, 4))
    return MOE_ERR_ALIGN;
  return MOE_OK;
}
// Whether [p, p + n) meets one of the batch's arrays.
bool meets_batch(const Span &s, const moe_batch &b) {
  return overlap(s, {b.q_start, 4 * ((uint64_t)b.n_seqs + 1)}) || overlap(s, {b.kv_len, 4 * (uint64_t)b.n_rows}) ||
         overlap(s, {b.table, 4 * (uint64_t)b.n_rows * b.table_cols}) || overlap(s, {b.row, 4 * (uint64_t)b.n_seqs});
}

PagedKv dev_kv(const moe_paged_kv &kv) {
  PagedKv p{};
  p.k = static_cast<uint16_t *>(kv.k);
  p.v = static_cast<uint16_t *>(kv.v);
  p.ps = kv.page_stride;
  p.ts = kv.token_stride;
  p.hs = kv.head_stride;
  p.n_pages = kv.n_pages;
  p.page_shift = __builtin_ctz((unsigned)kv.page_size);
  p.n_kv = kv.n_kv_heads;
  p.dim = kv.head_dim;
  p.fp16 = kv.dtype == MOE_FP16;
  return p;
}
Batch dev_batch(const moe_batch &b) {
  return Batch{b.q_start, b.kv_len, b.table, b.row, b.n_seqs, b.n_rows, b.table_cols};
}

moe_status check_attn_sizes(int64_t T, int32_t n_seqs, int64_t max_q, int64_t max_kv, int32_t n_heads,
                            const moe_paged_kv &kv) {
  if (T < 0 || T > kMaxTokens) return MOE_ERR_TOKENS;
  if (n_seqs < 1 || n_seqs > 65535 || max_q < 0 || max_kv < 0) return MOE_ERR_SHAPE;
  if (n_heads < 1 || n_heads > 4096 || n_heads % kv.n_kv_heads) return MOE_ERR_SHAPE;
  // (launches of at most 2^24 workgroups)
  if (T * n_heads > int64_t(1) << 29 || (int64_t)n_seqs * kv.n_kv_heads > int64_t(1) << 22) return MOE_ERR_TOKENS;
  return MOE_OK;
}

AttnShape shape_of(int64_t T, int32_t n_seqs, int64_t max_q, int64_t max_kv, int32_t window, int32_t n_heads,
                   const moe_paged_kv &kv) {
  return attn_shape(T, n_seqs, std::min<int64_t>(max_q, kMaxTokens), std::min<int64_t>(max_kv, int64_t(1) << 30), window, n_heads,
                    kv.n_kv_heads, kv.head_dim);
}

bool meets_groups(const Span &s, const moe_prefix_groups *g) {
  return g && (overlap(s, {g->group_start, 4 * ((uint64_t)g->n_groups + 1)}) || overlap(s, {g->prefix_len, 4 * (uint64_t)g->n_groups}));
}

// What moe_paged_attn and moe_prefix_attn (groups not null) share behind the checks of sizes; shape()
// gives the launch's.
template <class F>
moe_status attn_call(const moe_paged_kv &kv, const moe_batch &batch, const moe_prefix_groups *groups, int64_t T, const moe_heads *q,
                     int32_t n_heads, const moe_heads *out, float *lse, float scale, int32_t window, uint32_t flags, F shape,
                     void *workspace, size_t workspace_bytes, hipStream_t stream) {
  moe_status st;
  if (flags & ~MOE_ATTN_FULL) return MOE_ERR_SHAPE;
  const float scale_log2 = scale * 1.44269504088896341f;  // scores are kept as base-2 exponents
  if (window < 0 || (window > 0 && (flags & MOE_ATTN_FULL)) || !std::isfinite(scale_log2)) return MOE_ERR_SHAPE;
  if (T == 0) return MOE_OK;
  if ((st = check_heads(q)) != MOE_OK || (st = check_heads(out)) != MOE_OK) return st;
  if (!aligned(lse, 4)) return MOE_ERR_ALIGN;
  const int64_t D = kv.head_dim;
  if (!heads_distinct(*out, T, n_heads, D)) return MOE_ERR_SHAPE;
  const AttnShape sh = shape();
  if (sh.ws_bytes > 0 && (!workspace || workspace_bytes < sh.ws_bytes)) return MOE_ERR_WORKSPACE;
  if (sh.ws_bytes > 0 && !aligned(workspace, 256)) return MOE_ERR_ALIGN;
  const Span sq = span(*q, T, n_heads, D), ck = kv_span(kv, kv.k), cv = kv_span(kv, kv.v);
  const Span so = span(*out, T, n_heads, D), sl{lse, 4 * (uint64_t)T * n_heads}, sw{workspace, sh.ws_bytes};
  if (heads_overlap(*out, n_heads, *q, n_heads, T, D)) return MOE_ERR_ALIAS;
  if (overlap(sl, sq) || overlap(sw, sq) || overlap(so, sl) || overlap(so, sw) || overlap(sl, sw)) return MOE_ERR_ALIAS;
  for (const Span &w : {so, sl, sw})
    if (overlap(w, ck) || overlap(w, cv) || meets_batch(w, batch) || meets_groups(w, groups)) return MOE_ERR_ALIAS;
  if ((st = device_ok()) != MOE_OK) return st;
  AttnArgs a{};
  a.kv = dev_kv(kv);
  a.b = dev_batch(batch);
  a.q = dev_heads(*q);
  a.out = dev_heads(*out);
  a.lse = lse;
  a.part = static_cast<float *>(workspace);
  a.stats = reinterpret_cast<AttnStats *>(static_cast<char *>(workspace) + sh.off_stats);
  a.T = (int)T;
  a.H = n_heads;
  a.G = n_heads / kv.n_kv_heads;
  a.rows = sh.rows;
  a.tiles = sh.tiles;
  a.splits = sh.splits;
  a.split_blocks = sh.split_blocks;
  a.wgs = sh.wgs;
  a.join_rows = sh.join_rows;
  a.rec = reinterpret_cast<AttnRec *>(static_cast<char *>(workspace) + sh.off_rec);
  a.window = window;
  a.full = flags & MOE_ATTN_FULL;
  a.scale_log2 = scale_log2;
  if (groups) {
    a.group_start = groups->group_start;
    a.prefix_len = groups->prefix_len;
    a.n_groups = groups->n_groups;
    a.p_tiles = sh.p_tiles;
    a.p_splits = sh.p_splits;
    a.p_blocks = sh.p_blocks;
  }
  return launch_paged_attn(a, stream) == hipSuccess ? MOE_OK : MOE_ERR_HIP;
}

moe_status check_prefix_sizes(int64_t T, int32_t n_seqs, int32_t n_groups, int64_t max_q, int64_t max_prefix, int64_t max_suffix,
                              int32_t n_heads, const moe_paged_kv &kv) {
  const moe_status st = check_attn_sizes(T, n_seqs, max_q, max_prefix, n_heads, kv);
  if (st != MOE_OK) return st;
  if (n_groups < 1 || n_groups > n_seqs || max_suffix < 0) return MOE_ERR_SHAPE;
  return T * n_heads > int64_t(1) << 20 ? MOE_ERR_TOKENS : MOE_OK;
}
AttnShape shape_of(int64_t T, int32_t n_seqs, int32_t n_groups, int64_t max_q, int64_t max_prefix, int64_t max_suffix,
                   int32_t n_heads, const moe_paged_kv &kv) {
  return prefix_shape(T, n_seqs, n_groups, std::min<int64_t>(max_q, kMaxTokens), std::min<int64_t>(max_prefix, int64_t(1) << 30),
                      std::min<int64_t>(max_suffix, int64_t(1) << 30), n_heads, kv.n_kv_heads, kv.head_dim);
}

// ------------------------------------------------------------------------ pages

moe_status check_pages(const moe_pages *p) {
  if (!p || !p->table || !p->len || !p->refs) return MOE_ERR_NULL;
  if (p->n_seqs < 1 || p->n_seqs > 65535 || p->table_cols < 1 || p->n_pages < 1 || p->n_pages > 1 << 26)
    return MOE_ERR_SHAPE;
  if (p->page_size < 1 || p->page_size > 65536 || (p->page_size & (p->page_size - 1))) return MOE_ERR_SHAPE;
  if ((int64_t)p->table_cols * p->page_size > int64_t(1) << 30 || (int64_t)p->n_seqs * p->table_cols >= int64_t(1) << 31)
    return MOE_ERR_SHAPE;
  if (!aligned(p->table, 4) || !aligned(p->len, 4) || !aligned(p->refs, 4)) return MOE_ERR_ALIGN;
  return MOE_OK;
}
moe_status check_memory(const moe_page_memory *m, int32_t n_pages) {
  if (!m || !m->base) return MOE_ERR_NULL;
  if (m->n_planes < 1 || m->n_planes > 65535 || m->page_bytes < 16 || m->page_bytes > int64_t(1) << 30) return MOE_ERR_SHAPE;
  if (m->plane_stride < 0 || m->page_stride < 0) return MOE_ERR_SHAPE;
  if (!aligned(m->base, 16) || m->plane_stride % 16 || m->page_stride % 16 || m->page_bytes % 16) return MOE_ERR_ALIGN;
  Dim d[2] = {{m->plane_stride, m->n_planes}, {m->page_stride, n_pages}};
  return distinct(d, 2, m->page_bytes) ? MOE_OK : MOE_ERR_SHAPE;
}
Span memory_span(const moe_page_memory &m, int32_t n_pages) {
  return Span{m.base, (uint64_t)((m.n_planes - 1) * m.plane_stride + (n_pages - 1) * m.page_stride + m.page_bytes)};
}
PageMem dev_memory(const moe_page_memory &m) {
  return PageMem{static_cast<uint8_t *>(m.base), m.plane_stride, m.page_stride, m.page_bytes, m.n_planes};
}

// The checks that every call on a pool shares, and its launch.  x, y: the requests' arrays.
moe_status pages_call(PageOp op, const moe_pages *in, const moe_pages *out, const moe_page_memory *mem, int32_t n,
                      const int32_t *x, const int32_t *y, int32_t *error, void *ws, size_t ws_bytes, hipStream_t stream) {
  const bool has_mem = op == PageOp::Fork || op == PageOp::Compact;
  const bool has_y = op == PageOp::Grow || op == PageOp::Fork;
  moe_status st = check_pages(in);
  if (st != MOE_OK || (st = check_pages(out)) != MOE_OK) return st;
  if (in->n_seqs != out->n_seqs || in->table_cols != out->table_cols || in->n_pages != out->n_pages ||
      in->page_size != out->page_size)
    return MOE_ERR_SHAPE;
  if (has_mem && (st = check_memory(mem, in->n_pages)) != MOE_OK) return st;
  if (n < 0 || n > in->n_seqs) return MOE_ERR_SHAPE;
  if (!error || (n > 0 && (!x || (has_y && !y)))) return MOE_ERR_NULL;
  if (!aligned(error, 4) || !aligned(x, 4) || !aligned(y, 4)) return MOE_ERR_ALIGN;
  const PageWs w = page_ws(in->n_seqs, in->n_pages, n);
  if (!ws || ws_bytes < w.total) return MOE_ERR_WORKSPACE;
  if (!aligned(ws, 256)) return MOE_ERR_ALIGN;
  const uint64_t nt = 4 * (uint64_t)in->n_seqs * in->table_cols, nl = 4 * (uint64_t)in->n_seqs, nr = 4 * (uint64_t)in->n_pages;
  const Span ti{in->table, nt}, li{in->len, nl}, ri{in->refs, nr}, to{out->table, nt}, lo{out->len, nl}, ro{out->refs, nr};
  const bool same = in->table == out->table && in->len == out->len && in->refs == out->refs;
  const Span sx{n ? x : nullptr, 4 * (uint64_t)n}, sy{n && has_y ? y : nullptr, 4 * (uint64_t)n}, se{error, 4}, sw{ws, w.total};
  const Span sm = has_mem ? memory_span(*mem, in->n_pages) : Span{nullptr, 0};
  // everything apart from each other, but the pools where they are one
  const Span all[] = {to, lo, ro, se, sw, sm, sx, sy, ti, li, ri};
  const int n_all = same ? 8 : 11, writes = 6;
  for (int i = 0; i < writes; ++i)
    for (int j = i + 1; j < n_all; ++j)
      if (overlap(all[i], all[j])) return MOE_ERR_ALIAS;
  if ((st = device_ok()) != MOE_OK) return st;
  if (same && n == 0 && op != PageOp::Compact) return MOE_OK;
  PageArgs a{};
  a.in = Pages{in->table, in->len, in->refs};
  a.out = Pages{out->table, out->len, out->refs};
  if (has_mem) a.mem = dev_memory(*mem);
  a.n_seqs = in->n_seqs;
  a.cols = in->table_cols;
  a.n_pages = in->n_pages;
  a.page_shift = __builtin_ctz((unsigned)in->page_size);
  a.n = n;
  a.a = x;
  a.b = y;
  a.error = error;
  auto at = [&](size_t o) { return reinterpret_cast<int32_t *>(static_cast<char *>(ws) + o); };
  a.hdr = at(0);
  a.free_n = at(w.free_n);
  a.bad = at(w.bad);
  a.base = at(w.base);
  a.col = at(w.col);
  a.longer = at(w.longer);
  a.fresh = at(w.fresh);
  a.moved = at(w.moved);
  return launch_pages(op, a, stream) == hipSuccess ? MOE_OK : MOE_ERR_HIP;
}

}  // namespace

extern "C" {

moe_status moe_rope_freqs(int32_t rot_dim, double base, moe_rope_scaling scaling, double factor, int64_t trained,
                          double *out, float *mscale) {
  if (!out || !mscale) return MOE_ERR_NULL;
  if (rot_dim < 2 || rot_dim > 256 || rot_dim % 2) return MOE_ERR_SHAPE;
  if (!(base > 1.0) || !std::isfinite(base)) return MOE_ERR_SHAPE;
  if ((int)scaling < MOE_ROPE_NONE || (int)scaling > MOE_ROPE_YARN) return MOE_ERR_SHAPE;
  if (scaling != MOE_ROPE_NONE && (!(factor >= 1.0) || !std::isfinite(factor))) return MOE_ERR_SHAPE;
  if (scaling == MOE_ROPE_YARN && trained < 1) return MOE_ERR_SHAPE;
  if (scaling == MOE_ROPE_NTK) {
    if (rot_dim < 4) return MOE_ERR_SHAPE;
    base *= std::pow(factor, (double)rot_dim / (rot_dim - 2));
  }
  constexpr double kTwoPi = 6.283185307179586477;
  for (int i = 0; i < rot_dim / 2; ++i) {
    double f = std::pow(base, -2.0 * i / rot_dim);
    if (scaling == MOE_ROPE_LINEAR) f /= factor;
    if (scaling == MOE_ROPE_YARN) {
      const double turns = (double)trained * f / kTwoPi;
      const double keep = std::min(1.0, std::max(0.0, (turns - 1.0) / 31.0));
      f = f * keep + f / factor * (1.0 - keep);
    }
    out[i] = f;
  }
  *mscale = scaling == MOE_ROPE_YARN ? (float)(0.1 * std::log(factor) + 1.0) : 1.0f;
  return MOE_OK;
}

moe_status moe_rope_append(const moe_paged_kv *kv, const moe_batch *batch, int64_t T, const moe_heads *q,
                           const moe_heads *q_out, int32_t n_heads, const moe_heads *k, const moe_heads *v,
                           const int32_t *pos, const double *inv_freq, int32_t rot_dim, float mscale, uint32_t flags,
                           hipStream_t stream) {
  if (!kv || !k || !v) return MOE_ERR_NULL;
  if ((k->p == nullptr) != (v->p == nullptr)) return MOE_ERR_NULL;
  const bool append = k->p != nullptr;
  moe_status st = check_kv(kv, append);
  if (st != MOE_OK) return st;
  if ((st = check_batch(batch, kv->page_size)) != MOE_OK) return st;
  if (T < 0 || T > kMaxTokens) return MOE_ERR_TOKENS;
  const int64_t D = kv->head_dim, hk = append ? kv->n_kv_heads : 0;
  if (n_heads < 0 || n_heads > 4096 || rot_dim < 0 || rot_dim > D || rot_dim % 2) return MOE_ERR_SHAPE;
  if (flags & ~MOE_ROPE_INTERLEAVED) return MOE_ERR_SHAPE;
  if (rot_dim > 0 && !inv_freq) return MOE_ERR_NULL;
  if (!aligned(inv_freq, 8) || !aligned(pos, 4)) return MOE_ERR_ALIGN;
  if (T > 0 && n_heads > 0) {
    if ((st = check_heads(q)) != MOE_OK || (st = check_heads(q_out)) != MOE_OK) return st;
    if (!heads_distinct(*q_out, T, n_heads, D)) return MOE_ERR_SHAPE;
  }
  if (T > 0 && append && ((st = check_heads(k)) != MOE_OK || (st = check_heads(v)) != MOE_OK)) return st;
  if (T == 0) return MOE_OK;
  const Span ck = append ? kv_span(*kv, kv->k) : Span{}, cv = append ? kv_span(*kv, kv->v) : Span{};
  const Span sk = append ? span(*k, T, hk, D) : Span{}, sv = append ? span(*v, T, hk, D) : Span{};
  const Span spos{pos, 4 * (uint64_t)T}, sf{inv_freq, 4 * (uint64_t)rot_dim};
  if (append && planes_overlap(*kv)) return MOE_ERR_ALIAS;
  Span written[3] = {ck, cv, {}};
  for (int i = 0; i < 2; ++i)
    if (overlap(written[i], sk) || overlap(written[i], sv)) return MOE_ERR_ALIAS;
  if (n_heads > 0) {
    const Span so = span(*q_out, T, n_heads, D), sq = span(*q, T, n_heads, D);
    written[2] = so;
    const bool same = q->p == q_out->p && q->token_stride == q_out->token_stride && q->head_stride == q_out->head_stride;
    if (!same && heads_overlap(*q_out, n_heads, *q, n_heads, T, D)) return MOE_ERR_ALIAS;
    if (append && (heads_overlap(*q_out, n_heads, *k, hk, T, D) || heads_overlap(*q_out, n_heads, *v, hk, T, D)))
      return MOE_ERR_ALIAS;
    for (int i = 0; i < 2; ++i)
      if (overlap(written[i], so) || overlap(written[i], sq)) return MOE_ERR_ALIAS;
  }
  for (const Span &w : written)
    if (overlap(w, spos) || overlap(w, sf) || meets_batch(w, *batch)) return MOE_ERR_ALIAS;
  if ((st = device_ok()) != MOE_OK) return st;
  RopeArgs a{};
  a.kv = dev_kv(*kv);
  a.b = dev_batch(*batch);
  if (n_heads > 0) {
    a.q = dev_heads(*q);
    a.qo = dev_heads(*q_out);
  }
  a.k = dev_heads(*k);
  a.v = dev_heads(*v);
  a.pos = pos;
  a.freq = inv_freq;
  a.T = (int)T;
  a.H = n_heads;
  a.R = rot_dim;
  a.mscale = mscale;
  a.interleaved = flags & MOE_ROPE_INTERLEAVED;
  return launch_rope_append(a, stream) == hipSuccess ? MOE_OK : MOE_ERR_HIP;
}

moe_status moe_paged_attn_workspace(const moe_paged_kv *kv, int64_t T, int32_t n_seqs, int64_t max_q, int64_t max_kv,
                                    int32_t n_heads, int32_t window, size_t *bytes) {
  if (!bytes) return MOE_ERR_NULL;
  moe_status st = check_kv(kv, false);
  if (st != MOE_OK) return st;
  if ((st = check_attn_sizes(T, n_seqs, max_q, max_kv, n_heads, *kv)) != MOE_OK) return st;
  if (window < 0) return MOE_ERR_SHAPE;
  *bytes = shape_of(T, n_seqs, max_q, max_kv, window, n_heads, *kv).ws_bytes;
  return MOE_OK;
}

moe_status moe_paged_attn(const moe_paged_kv *kv, const moe_batch *batch, int64_t T, int64_t max_q, int64_t max_kv,
                          const moe_heads *q, int32_t n_heads, const moe_heads *out, float *lse, float scale,
                          int32_t window, uint32_t flags, void *workspace, size_t workspace_bytes, hipStream_t stream) {
  moe_status st = check_kv(kv, true);
  if (st != MOE_OK) return st;
  if ((st = check_batch(batch, kv->page_size)) != MOE_OK) return st;
  if ((st = check_attn_sizes(T, batch->n_seqs, max_q, max_kv, n_heads, *kv)) != MOE_OK) return st;
  return attn_call(*kv, *batch, nullptr, T, q, n_heads, out, lse, scale, window, flags,
                   [&] { return shape_of(T, batch->n_seqs, max_q, max_kv, window, n_heads, *kv); }, workspace, workspace_bytes,
                   stream);
}

moe_status moe_prefix_attn_workspace(const moe_paged_kv *kv, int64_t T, int32_t n_seqs, int32_t n_groups, int64_t max_q,
                                     int64_t max_prefix, int64_t max_suffix, int32_t n_heads, size_t *bytes) {
  if (!bytes) return MOE_ERR_NULL;
  moe_status st = check_kv(kv, false);
  if (st != MOE_OK) return st;
  if ((st = check_prefix_sizes(T, n_seqs, n_groups, max_q, max_prefix, max_suffix, n_heads, *kv)) != MOE_OK) return st;
  *bytes = shape_of(T, n_seqs, n_groups, max_q, max_prefix, max_suffix, n_heads, *kv).ws_bytes;
  return MOE_OK;
}

moe_status moe_prefix_attn(const moe_paged_kv *kv, const moe_batch *batch, const moe_prefix_groups *groups, int64_t T,
                           int64_t max_q, int64_t max_prefix, int64_t max_suffix, const moe_heads *q, int32_t n_heads,
                           const moe_heads *out, float *lse, float scale, uint32_t flags, void *workspace,
                           size_t workspace_bytes, hipStream_t stream) {
  moe_status st = check_kv(kv, true);
  if (st != MOE_OK) return st;
  if ((st = check_batch(batch, kv->page_size)) != MOE_OK) return st;
  if (!groups || !groups->group_start || !groups->prefix_len) return MOE_ERR_NULL;
  if (!aligned(groups->group_start, 4) || !aligned(groups->prefix_len, 4)) return MOE_ERR_ALIGN;
  if ((st = check_prefix_sizes(T, batch->n_seqs, groups->n_groups, max_q, max_prefix, max_suffix, n_heads, *kv)) != MOE_OK) return st;
  return attn_call(*kv, *batch, groups, T, q, n_heads, out, lse, scale, 0, flags,
                   [&] { return shape_of(T, batch->n_seqs, groups->n_groups, max_q, max_prefix, max_suffix, n_heads, *kv); },
                   workspace, workspace_bytes, stream);
}

moe_status moe_gdn_step(int32_t R, int32_t n_kheads, int32_t n_vheads, int32_t d_k, int32_t d_v, const void *q,
                        const void *k, const void *v, const float *alpha, const float *beta, float *state,
                        int32_t n_slots, const int32_t *slot, void *out, hipStream_t stream) {
  if (R < 0) return MOE_ERR_TOKENS;
  if (d_k != kGdnDim || d_v != kGdnDim) return MOE_ERR_SHAPE;
  if (n_kheads < 1 || n_vheads < 1 || n_vheads > 4096 || n_vheads % n_kheads != 0 || n_slots < 1) return MOE_ERR_SHAPE;
  if ((int64_t)R * n_vheads > int64_t(1) << 20) return MOE_ERR_TOKENS;
  if (!state) return MOE_ERR_NULL;
  if (R > 0 && (!q || !k || !v || !alpha || !beta || !slot || !out)) return MOE_ERR_NULL;
  if (!aligned(state, 16)) return MOE_ERR_ALIGN;
  if (R == 0) return MOE_OK;
  if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(alpha, 4) || !aligned(beta, 4) ||
      !aligned(slot, 4) || !aligned(out, 2))
    return MOE_ERR_ALIGN;
  const uint64_t nqk = (uint64_t)R * n_kheads * kGdnDim * 2, nv = (uint64_t)R * n_vheads * kGdnDim * 2;
  const uint64_t ng = (uint64_t)R * n_vheads * 4;
  const Span so{out, nv}, ss{state, (uint64_t)n_slots * n_vheads * kGdnDim * kGdnDim * 4};
  for (const Span &w : {so, ss})
    for (const Span &r : {Span{q, nqk}, Span{k, nqk}, Span{v, nv}, Span{alpha, ng}, Span{beta, ng},
                          Span{slot, 4 * (uint64_t)R}})
      if (overlap(w, r)) return MOE_ERR_ALIAS;
  if (overlap(so, ss)) return MOE_ERR_ALIAS;
  const moe_status st = device_ok();
  if (st != MOE_OK) return st;
  GdnStepArgs a{};
  a.q = static_cast<const uint16_t *>(q);
  a.k = static_cast<const uint16_t *>(k);
  a.v = static_cast<const uint16_t *>(v);
  a.alpha = alpha;
  a.beta = beta;
  a.state = state;
  a.slot = slot;
  a.out = static_cast<uint16_t *>(out);
  a.R = R;
  a.hk = n_kheads;
  a.hv = n_vheads;
  a.n_slots = n_slots;
  return launch_gdn_step(a, stream) == hipSuccess ? MOE_OK : MOE_ERR_HIP;
}

moe_status moe_pages_workspace(const moe_pages *pages, int32_t n, size_t *bytes) {
  if (!pages || !bytes) return MOE_ERR_NULL;
  if (pages->n_seqs < 1 || pages->n_seqs > 65535 || pages->n_pages < 1 || pages->n_pages > 1 << 26) return MOE_ERR_SHAPE;
  if (n < 0 || n > pages->n_seqs) return MOE_ERR_SHAPE;
  *bytes = page_ws(pages->n_seqs, pages->n_pages, n).total;
  return MOE_OK;
}

moe_status moe_pages_grow(const moe_pages *in, const moe_pages *out, int32_t n, const int32_t *seqs,
                          const int32_t *tokens, int32_t *error, void *workspace, size_t workspace_bytes,
                          hipStream_t stream) {
  return pages_call(PageOp::Grow, in, out, nullptr, n, seqs, tokens, error, workspace, workspace_bytes, stream);
}

moe_status moe_pages_fork(const moe_pages *in, const moe_pages *out, const moe_page_memory *mem, int32_t n,
                          const int32_t *src, const int32_t *dst, int32_t *error, void *workspace,
                          size_t workspace_bytes, hipStream_t stream) {
  return pages_call(PageOp::Fork, in, out, mem, n, src, dst, error, workspace, workspace_bytes, stream);
}

moe_status moe_pages_free(const moe_pages *in, const moe_pages *out, int32_t n, const int32_t *seqs, int32_t *error,
                          void *workspace, size_t workspace_bytes, hipStream_t stream) {
  return pages_call(PageOp::Free, in, out, nullptr, n, seqs, nullptr, error, workspace, workspace_bytes, stream);
}

moe_status moe_pages_compact(const moe_pages *in, const moe_pages *out, const moe_page_memory *mem, int32_t *error,
                             void *workspace, size_t workspace_bytes, hipStream_t stream) {
  return pages_call(PageOp::Compact, in, out, mem, 0, nullptr, nullptr, error, workspace, workspace_bytes, stream);
}

moe_status moe_pages_copy(const moe_page_memory *mem, int32_t n_pages, int32_t n, const int32_t *src,
                          const int32_t *dst, hipStream_t stream) {
  if (n_pages < 1 || n_pages > 1 << 26 || n < 0 || n > 1 << 20) return MOE_ERR_SHAPE;
  moe_status st = check_memory(mem, n_pages);
  if (st != MOE_OK) return st;
  if (n == 0) return MOE_OK;
  if (!src || !dst) return MOE_ERR_NULL;
  if (!aligned(src, 4) || !aligned(dst, 4)) return MOE_ERR_ALIGN;
  const Span sm = memory_span(*mem, n_pages);
  if (overlap(sm, {src, 4 * (uint64_t)n}) || overlap(sm, {dst, 4 * (uint64_t)n})) return MOE_ERR_ALIAS;
  if ((st = device_ok()) != MOE_OK) return st;
  return launch_pages_copy(dev_memory(*mem), n_pages, n, src, dst, stream) == hipSuccess ? MOE_OK : MOE_ERR_HIP;
}

moe_status moe_pages_check(const int32_t *error, hipStream_t stream) {
  if (!error) return MOE_ERR_NULL;
  int32_t e = 0;
  if (hipMemcpyAsync(&e, error, 4, hipMemcpyDeviceToHost, stream) != hipSuccess || hipStreamSynchronize(stream) != hipSuccess)
    return MOE_ERR_HIP;
  return (moe_status)e;
}

}  // extern "C"
