// Launch interfaces of the serving operators: rotary append, paged attention, gated delta
// steps (host side calls these from serve_api.cpp), norm, 4-bit projections and sampling
// (from step_api.cpp).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <atomic>

namespace moe {

// Sets the LDS limit of a kernel, once for each device (the attribute belongs to the device).
template <class K>
hipError_t allow_lds(K k, int lds, std::atomic<uint64_t> &done) {
  int dev = 0;
  hipError_t e = hipGetDevice(&dev);
  if (e != hipSuccess) return e;
  if (dev <= 63 && done.load(std::memory_order_relaxed) >> dev & 1) return hipSuccess;
  e = hipFuncSetAttribute((const void *)k, hipFuncAttributeMaxDynamicSharedMemorySize, lds);
  if (e == hipSuccess && dev <= 63) done.fetch_or(uint64_t(1) << dev, std::memory_order_relaxed);
  return e;
}

struct Heads {  // [token][head][head_dim] with strides in elements
  uint16_t *p;
  int64_t ts, hs;
};

struct PagedKv {
  uint16_t *k, *v;
  int64_t ps, ts, hs;  // page, token and head strides in elements
  int n_pages, page_shift, n_kv, dim;
  bool fp16;
};

struct Batch {
  const int32_t *q_start, *kv_len, *table, *row;
  int n_seqs, n_rows, cols;
};

struct RopeArgs {
  PagedKv kv;
  Batch b;
  Heads q, qo, k, v;  // k.p null: nothing is appended
  const int32_t *pos;
  const double *freq;
  int T, H, R;
  float mscale;
  bool interleaved;
};
hipError_t launch_rope_append(const RopeArgs &a, hipStream_t s);

constexpr int kAttnRows = 16;   // query rows (token x head of a group) of a small tile
constexpr int kAttnTile = 128;  // query rows of a large tile: four waves of 32
constexpr int kAttnKeys = 32;   // keys of one block

// Of a partial output: reference (base-2 exponent), sums of the rounded and of the unrounded
// weights.
struct AttnStats {
  float m, l, e, pad;
};

// A segment (row tile and key/value head) whose keys n consecutive workgroups share.
struct AttnRec {
  int n, t0, r0, nr, kvh;
};

struct AttnArgs {
  PagedKv kv;
  Batch b;
  Heads q, out;
  float *lse;      // [T][H] or null
  float *part;     // unnormalised partial outputs: [T * H][splits][dim], small tiles [wgs][2][16][dim]
  AttnStats *stats;  // of each
  int T, H, G;     // G: query heads of one key/value head
  int rows;        // rows of a tile: kAttnRows or kAttnTile
  int tiles;       // bound on the number of row tiles
  int splits, split_blocks;
  int wgs, join_rows;  // small tiles: workgroups, and rows that the join takes at once
  AttnRec *rec;        // [wgs]
  int window;
  bool full;
  float scale_log2;
  // shared prefixes (n_groups > 0): the first p_splits of the splits are of the prefixes
  const int32_t *group_start, *prefix_len;
  int n_groups, p_tiles, p_splits, p_blocks;
};
// What the launch is shaped by, from host-known sizes alone.
struct AttnShape {
  int rows, tiles, splits, split_blocks, wgs, join_rows, p_tiles, p_splits, p_blocks;
  size_t ws_bytes, off_stats, off_rec;
};
AttnShape attn_shape(int64_t T, int n_seqs, int64_t max_q, int64_t max_kv, int window, int H, int n_kv, int dim);
AttnShape prefix_shape(int64_t T, int n_seqs, int n_groups, int64_t max_q, int64_t max_prefix, int64_t max_suffix, int H, int n_kv,
                       int dim);
hipError_t launch_paged_attn(const AttnArgs &a, hipStream_t s);

struct GdnStepArgs {
  const uint16_t *q, *k, *v;
  const float *alpha, *beta;
  float *state;
  const int32_t *slot;
  uint16_t *out;
  int R, hk, hv, n_slots;
};
hipError_t launch_gdn_step(const GdnStepArgs &a, hipStream_t s);

// Paged cache bookkeeping (pages.hip).
struct Pages {
  int32_t *table, *len, *refs;
};
struct PageMem {
  uint8_t *base;
  int64_t plane, page, bytes;  // strides and size in bytes
  int n_planes;
};
constexpr int kPageGroup = 4096;  // pages whose free ones are counted by one workgroup

enum class PageOp { Grow, Fork, Free, Compact };

struct PageArgs {
  Pages in, out;
  PageMem mem;
  int n_seqs, cols, n_pages, page_shift;
  int n;               // requests
  const int32_t *a, *b;  // grow: sequences, tokens; fork: sources, destinations; free: sequences
  int32_t *error;
  // workspace
  int32_t *hdr;        // [0] status of the requests, [1] fresh pages needed, [2] pages that move
  int32_t *free_n;     // [groups] free pages of the group
  int32_t *bad;        // [requests, or sequences (compact)] a table entry lies outside the pool
  int32_t *base;       // [n + 1] fresh pages needed before the request
  int32_t *col, *longer;  // [n] grow: pages held before, length after
  int32_t *fresh;      // fork: [groups][kPageGroup] a group's first free pages; compact: [n_pages] free
                       // page by rank
  int32_t *moved;      // compact: [n_pages] page that moves, by rank from the pool's end
};
struct PageWs {
  size_t free_n, bad, base, col, longer, fresh, moved, total;
};
PageWs page_ws(int n_seqs, int n_pages, int n);
hipError_t launch_pages(PageOp op, const PageArgs &a, hipStream_t s);
hipError_t launch_pages_copy(const PageMem &m, int n_pages, int n, const int32_t *src, const int32_t *dst, hipStream_t s);

// Norm with the residual's addition (norm.hip).
struct Rows {  // [token][head][width], strides in elements
  void *p;
  int64_t ts, hs;
};
struct NormArgs {
  Rows x, r, sum, out;  // r.p, sum.p null: none
  const uint16_t *w;    // or null
  float *scale;         // 8-bit outputs: [rows][groups]
  int64_t rows;         // T * n
  int n, W, group;      // group: W where a row is one
  float offset, eps;
  int out_kind;         // 0: the input's type, 1: int8, 2: e4m3
  bool fp16, vec;       // vec: 16-byte rows
};
hipError_t launch_rms_norm(const NormArgs &a, hipStream_t s);

// Products of few rows with 4-bit weights (linear.hip).
enum class LinX { Bf16, Fp16, Int8 };
enum class LinOut { Bf16, Fp16, Fp32 };
struct LinArgs {
  const uint32_t *codes;
  const uint16_t *scale, *bias;
  const void *x;
  const float *xs;      // int8: [T][xs_cols]
  void *out;
  int64_t xld, old;     // strides of x's and out's rows in elements
  int64_t T;
  int n, k, cols;  // cols: workgroups that share a run of weights
  int xs_cols, xs_shift;  // a group of 64 has scale (group >> xs_shift), 31: the row's
  bool qbf16;
  LinX x_type;
  LinOut out_type;
};
hipError_t launch_linear(const LinArgs &a, hipStream_t s);

// Choice of tokens from logits (sample.hip).
constexpr int kSampleChunk = 4096;  // logits of one workgroup of the first kernel
constexpr int kSampleBins = 192;    // bins of a chunk's weights, an eighth of an octave each
// Of a chunk: its largest logit (times log2(e) / temperature) and the sum of its weights; for a
// temperature of 0 the largest logit's sort key and index.
struct SampleChunk {
  double top;
  uint64_t total, best;
};
// Of a row with filters: its bins, summed down to each, the bins of the first cut, and the tokens listed.
constexpr int kSampleList = 16384;
struct SampleRow {
  uint64_t mass[kSampleBins];
  uint32_t count[kSampleBins];
  int lo, hi;  // hi < lo: no cut
  int n;       // tokens that lie between the bins' bounds, of which the first kSampleList are listed
  int pad;
};
struct SampleArgs {
  const void *logits;
  int64_t ld;
  int type;  // 0: fp32, 1: bf16, 2: fp16
  const float *u, *temperature, *top_p, *min_p;
  const int32_t *top_k;
  int32_t *token;
  float *prob;
  int R, V, C, bits;  // C: chunks of a row; bits of a weight behind 1
  SampleChunk *chunk;  // [R][C]
  uint64_t *mass;      // [R][C][bins]
  uint32_t *count;     // [R][C][bins]
  SampleRow *row;      // [R]
  uint64_t *kept;      // [R][C] weight of a chunk's bins above the cut's
  uint64_t *list;      // [R][room]
  int room;            // min(V, kSampleList)
};
hipError_t launch_sample(const SampleArgs &a, hipStream_t s);

}  // namespace moe
