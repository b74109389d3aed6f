// Attention of a ragged batch of new tokens over the paged cache.
//
// Per query row: out = sum_j p_j v_j / sum_j p_j, p_j = exp(scale q.k_j - m), with a reference m,
// the sums and the output rescaled as keys go by (one pass over K and V).  Scores, m, sums and
// outputs are binary32; p_j is rounded to the cache's type to enter the matrix units.
//
// A query row is a (token, head) pair; the rows of one key/value head's group are packed into
// tiles, so the heads that share a key/value head share every load.  Keys go by in blocks of 32.
// Both products are computed transposed: S^T = K Q^T leaves a lane one query's scores, 4 keys
// at a time, and with the contraction index of P V ordered the same way those registers are
// P^T's operand as they are; V^T comes from ds_read_b64_tr_b16.
//
//   k_attn_tile  128 rows, four waves of 32 (v_mfma_f32_32x32x16), every wave all keys; blocks of
//                K and V in an LDS ring filled by direct-to-LDS loads.  Where tiles are few,
//                their keys are split over workgroups, joined by k_attn_join(_few).
//                Bound: matrix units (4 flops per row, visible key and element).  4096 tokens at
//                32K, 16/2 heads of 256: 1.77 to 1.82 ms by card, 1.16 to 1.13 PFLOP/s (a large library
//                product reaches 1.22; the same over zeros 1.35 ms: power); 4096 at 16K, 32/8 heads of
//                128, 1.04 ms (floor 0.79), and at 8K, 16/16 of 64, 0.186 ms (0.084): matrix units
//                busy for 69, 48 and 23 % of the cycles, vector units 44, 55 and 48.  24 chunks of 0 to
//                509 tokens, window 1024, 32/8 heads of 128, fp16: 0.127 ms, 0.64 PFLOP/s (masked
//                parts of blocks, an uneven last round).  One token at 4K: 12.0 us, a chain of
//                dependent loads and a second launch.  With PREFIX, rows of many sequences against
//                a prefix that they share, and each sequence's against the keys behind it, all in one
//                launch: 64 tokens, 16/2 heads of 256, up to 512 keys behind a prefix of 16384, 41.8 us
//                (38 and the join's 7 under the profiler), 17 GFLOP of the prefix's and 9 of short tiles.
//                0.95 us a block where a compute unit has one such tile, half of it the matrix units' (a ring of
//                three blocks, and so one workgroup a compute unit, takes as long a block and 50 us in all);
//                the rest is the start, a chain of loads (groups, batch, table, pages, keys), and 33 MB of partial
//                results.
//   k_attn_rows  16 rows, four waves sharing the keys out (v_mfma_f32_16x16x32); the keys of all
//                sequences cut into equal runs, joined by k_attn_join_runs.  For few rows over
//                many long sequences.  Bound: memory.  One token of 64 sequences up to 16K:
//                171 us, 5.0 TB/s (a copy reaches 5.2).
//
// Results of splits and runs are joined by their references, in fixed order.
#include <algorithm>

#include "paged.hpp"

#pragma clang fp contract(off)

namespace moe {

namespace {

typedef __attribute__((__vector_size__(4 * sizeof(float)))) float f32x4;
typedef __attribute__((__vector_size__(8 * sizeof(_Float16)))) _Float16 f16x8;
typedef __attribute__((__vector_size__(4 * sizeof(short)))) short s16x4;

constexpr int kThreads = 256, kWaves = 4;
constexpr int kMaxSplits = 256;
// workgroups of k_attn_tile that splits aim at: two a compute unit, three of narrow heads (heads of 64,
// 32 tokens of 8 sequences at 2K 19.1 us, 22.4 with two; of 128, 16 of 6 at 6K 30.6 and 28.6)
constexpr int tile_slots(int dim) { return dim == 64 ? 768 : 512; }
constexpr int kWhole = 7;        // blocks that are worth no second launch
constexpr int kMaxRuns = 1024;  // workgroups of k_attn_rows at most
// workgroups of k_attn_rows that fill the chip (registers allow 1, 2 or 3 on a compute unit)
constexpr int runs_of(int dim) { return dim == 256 ? 256 : dim == 128 ? 512 : 768; }
constexpr float kLn2 = 0.69314718055994531f;

template <bool F16>
__device__ __forceinline__ f32x4 mfma16(u32x4 a, u32x4 b, f32x4 c) {
  if constexpr (F16)
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}

// (lo, hi) rounded to nearest even and packed.
template <bool F16>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  if constexpr (F16) {
    typedef __attribute__((__vector_size__(2 * sizeof(_Float16)))) _Float16 f16x2;
    return __builtin_bit_cast(uint32_t, f16x2{(_Float16)lo, (_Float16)hi});
  }
  else
    return pack_bf16x2(lo, hi);
}
template <bool F16>
__device__ __forceinline__ float unpack(uint32_t w, bool hi) {
  const uint16_t v = (uint16_t)(hi ? w >> 16 : w & 0xffff);
  return F16 ? fp16_to_f32(v) : bf16_to_f32(v);
}
// c plus both values of a word
template <bool F16>
__device__ __forceinline__ float add2(uint32_t w, float c) {
  if constexpr (F16) {
    typedef __attribute__((__vector_size__(2 * sizeof(_Float16)))) _Float16 f16x2;
    return __builtin_amdgcn_fdot2(__builtin_bit_cast(f16x2, w), f16x2{(_Float16)1.0f, (_Float16)1.0f}, c, false);
  } else {
    return dot2_bf16(w, 0x3f803f80u, c);
  }
}
// fp16 holds numbers of 2^-14 to 2^15 with all their bits and none below 2^-25, and a row with one
// dominant key may have its value from keys far below that one.  So its weights are taken as 2^bias times
// what they are: the largest is 2^15 in k_attn_rows, and 2^11 to 2^15 in k_attn_tile, whose reference
// lags by up to 2^4.  Weights down to 2^-29 (2^-25) of the largest keep all bits, and 2^17 keys that
// are too small to be held make up 2^-23 (2^-19) of a row at most.  (With the largest weight at 1, or
// 2^8, all of 2^17 keys at e^-17.4 behind one at 0 were lost: 0.4 % of the row, 7 roundings of fp16.
// The shorter lag costs 0 to 4 %: 512 tokens at 8K, heads of 256, 94.3 -> 97.8 us, 24 ragged chunks,
// heads of 128, 122 -> 124.)  The factor is in all of a row's sums and cancels in its output.
constexpr float lag_of(bool f16) { return f16 ? 4.0f : 8.0f; }
constexpr float rows_bias(bool f16) { return f16 ? 15.0f : 0.0f; }
constexpr float tile_bias(bool f16) { return f16 ? 15.0f - lag_of(true) : 0.0f; }

// What is kept of a row besides its weighted sum of values: the reference (base-2 exponent), the
// sum of the rounded weights, which the values' sum is divided by (so that a weight's rounding
// only shifts the mean of the values), and that of the unrounded ones, for the log-sum-exp; both sums
// 2^bias times what they are.
struct Stats {
  float m, l, e;
};
__device__ __forceinline__ float lse_of(float m, float e, float bias) {
  return e == 0.0f ? -INFINITY : (m + (__log2f(e) - bias)) * kLn2;
}
__device__ __forceinline__ float reciprocal_of(float l) { return l == 0.0f ? 0.0f : 1.0f / l; }

// whether a value is an infinity or NaN
template <bool F16>
__device__ __forceinline__ bool nonfinite16(uint32_t w) {
  const uint32_t m = F16 ? 0x7c00u : 0x7f80u;
  return (w & m) == m;
}

__device__ __forceinline__ uint64_t tr_read(uint32_t lds) {
  return __builtin_bit_cast(uint64_t, __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                                          (__attribute__((address_space(3))) s16x4 *)(uintptr_t)lds));
}

// Maximum and sum over the four 16-lane groups (every lane gets its column's).
__device__ __forceinline__ float groups_max(float v) {
  auto a = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  v = fmaxf(__uint_as_float(a[0]), __uint_as_float(a[1]));
  auto b = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return fmaxf(__uint_as_float(b[0]), __uint_as_float(b[1]));
}
__device__ __forceinline__ float groups_sum(float v) {
  auto a = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  v = __uint_as_float(a[0]) + __uint_as_float(a[1]);
  auto b = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return __uint_as_float(b[0]) + __uint_as_float(b[1]);
}

template <int N>
__device__ __forceinline__ void wait_vm() {
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}
__device__ __forceinline__ void wait_lds() { asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory"); }

// 16-byte chunk c of LDS row r lies at chunk c ^ swz(r).  K is read 16 rows at a time at one
// chunk, V four rows in a row at four chunks in a row: swz is different for 16 rows (8 of rows of
// 128 bytes, of which two lie side by side over the banks), and takes four consecutive rows to
// four different groups of four chunks, so either read touches every bank once.  (With swz = r,
// whose four consecutive rows stay in one group, 60 % of the LDS cycles were conflicts.)
// It is linear in the bits of r.
template <int D>
__device__ __forceinline__ int swz(int r) {
  return D == 64 ? (r & 2) << 1 | (r >> 2 & 3) : (r & 3) << 2 | (r >> 2 & 3);
}

// Single page table entries are read as constants, by the scalar unit.
typedef const __attribute__((address_space(4))) int32_t *TableRow;

// The page of the 16 keys from `key` on, or -1.
__device__ __forceinline__ int page_at(const AttnArgs &a, TableRow row, int key) {
  const int col = __builtin_amdgcn_readfirstlane(key >> a.kv.page_shift);
  const int page = row[min(col, a.b.cols - 1)];
  return __builtin_amdgcn_readfirstlane(col < a.b.cols && (unsigned)page < (unsigned)a.kv.n_pages ? page : -1);
}
__device__ __forceinline__ TableRow table_row(const AttnArgs &a, int row) {
  return (TableRow)(uintptr_t)uniform_ptr(a.b.table + (int64_t)max(row, 0) * a.b.cols);
}

// A tile's place in its sequence: its query rows and the keys they see.
struct Tile {
  int row;            // of the table, -1: none
  int t0, n;          // first token, number of new tokens
  int r0, nr;         // first row (token * G + head) and rows of the tile
  int64_t first;      // position of the sequence's first new token
  int len;            // keys stored: min(kv_len, columns * page size)
  int lo, hi;         // keys that any row of the tile sees lie in [lo, hi)
  bool full;          // every row sees every key in there
};

// A sequence of the batch: first token, new tokens (0 where the numbers are no batch: nothing is
// touched then), table row (or -1) and length.
struct Seq {
  int t0, n, row, total;
};
__device__ __forceinline__ Seq read_seq(const AttnArgs &a, int s) {
  const Batch &b = a.b;
  Seq q;
  q.t0 = b.q_start[s];
  const int t1 = b.q_start[s + 1];
  q.row = batch_row(b, s);
  const int len = b.kv_len[max(q.row, 0)];
  q.total = q.row < 0 ? 0 : len;
  q.n = q.t0 < 0 || t1 > a.T ? 0 : max(t1 - q.t0, 0);
  return q;
}

// The tile of `rows` rows from r0 of a sequence on.  Returns whether there are any.
__device__ __forceinline__ bool set_tile(const AttnArgs &a, const Seq &q, int64_t r0, int rows, Tile &t) {
  t.t0 = q.t0;
  t.n = q.n;
  if (r0 < 0 || r0 >= (int64_t)t.n * a.G) return false;
  t.r0 = (int)r0;
  t.nr = min(rows, t.n * a.G - t.r0);
  t.row = q.row;
  t.full = a.full;
  t.first = (int64_t)q.total - t.n;
  t.len = min(max(q.total, 0), a.b.cols << a.kv.page_shift);
  const int64_t p0 = t.first + t.r0 / a.G, p1 = t.first + (t.r0 + t.nr - 1) / a.G;
  int64_t lo = 0, hi = t.len;
  if (!a.full && p1 + 1 < hi) hi = p1 + 1;
  if (a.window && p0 - a.window + 1 > lo) lo = p0 - a.window + 1;
  t.hi = (int)max(hi, (int64_t)0);
  t.lo = (int)min(lo, (int64_t)t.hi);
  return true;
}

__device__ __forceinline__ Seq readlane_seq(const Seq &q, int l) {
  return Seq{__builtin_amdgcn_readlane(q.t0, l), __builtin_amdgcn_readlane(q.n, l), __builtin_amdgcn_readlane(q.row, l),
             __builtin_amdgcn_readlane(q.total, l)};
}

// The x-th tile of `rows`-row tiles to be taken, out of a.tiles or fewer: of a sequence the last
// ones, which see most keys, first.
__device__ __forceinline__ bool find_tile(const AttnArgs &a, int x, int rows, Tile &t, int &seq) {
  const Batch &b = a.b;
  if (b.n_seqs > 1 && b.n_seqs <= 64) {
    // Every sequence in a lane, so that a tile's is not read once more (a step in the chain of
    // loads), and the longer ones first, so that short tiles fill the last round: 30 chunks of up
    // to 300 tokens at up to 5000, 32/8 heads of 128, 274 us (328 in the order they come); one token
    // of 16 sequences at 500 12.4 (13.0).  One sequence has nothing of either: 0.4 us more here.
    const int lane = threadIdx.x & 63;
    const Seq mine = read_seq(a, min(lane, b.n_seqs - 1));
    const int tiles = lane < b.n_seqs ? (int)(((int64_t)mine.n * a.G + rows - 1) / rows) : 0;
    const float seen = (float)(a.window ? min((int64_t)mine.total, (int64_t)a.window + mine.n) : mine.total);
    const bool longer = 2.0f * seen >= wave_max(tiles > 0 ? seen : 0.0f);
    int upto = wave_incl_scan(longer ? tiles : 0);
    uint64_t has = __ballot(upto > x);
    if (!has) {
      x -= __builtin_amdgcn_readlane(upto, 63);
      upto = wave_incl_scan(longer ? 0 : tiles);
      has = __ballot(upto > x);
      if (!has) return false;
    }
    const int s = seq = __builtin_ctzll(has);
    return set_tile(a, readlane_seq(mine, s), (int64_t)(__builtin_amdgcn_readlane(upto, s) - 1 - x) * rows, rows, t);
  }
  // Sequence b's tiles start at floor(q_start[b] G / rows) + b, which leaves room for
  // ceil(n_b G / rows) of them, so no list of tiles is needed
  x = a.tiles - 1 - x;
  const int s = seq = wave_find(b.n_seqs, x, [&](int i) { return (int64_t)b.q_start[i] * a.G / rows + i; });
  const Seq q = read_seq(a, s);
  return set_tile(a, q, ((int64_t)x - ((int64_t)q.t0 * a.G / rows + s)) * rows, rows, t);
}

// ------------------------------------------------------------ tiles of shared prefixes

// In the prefix form a tile is one of a group's prefix -- rows of all its sequences' tokens, which are
// consecutive, against the keys that these share -- or one of a sequence's suffix, whose keys start
// behind its group's prefix.  Workgroups: first the prefixes' (tiles x key/value heads x splits), then
// the suffixes'.
struct Work {
  int tile, kvh, split, per;  // per: blocks of a split
  int slot;                   // of the row's partial results
  bool prefix;
};
__device__ __forceinline__ Work work_of(const AttnArgs &a, int x) {
  Work w;
  const int n_kv = a.kv.n_kv, first = a.p_tiles * n_kv * a.p_splits;
  w.prefix = x < first;
  if (w.prefix) {
    // The tiles that share keys follow each other at a distance of 8 workgroups, so that one XCD's cache
    // brings these keys once.
    const int parts = n_kv * a.p_splits, whole = parts / 8 * 8 * a.p_tiles;
    int part;
    if (x < whole) {
      const int y = x / 8;
      w.tile = y % a.p_tiles;
      part = y / a.p_tiles * 8 + x % 8;
    } else {
      const int rest = parts % 8, y = x - whole;
      w.tile = y / rest;
      part = parts / 8 * 8 + y % rest;
    }
    w.kvh = part % n_kv;
    w.split = part / n_kv;
    w.per = a.p_blocks;
    w.slot = w.split;
  } else {
    x -= first;
    w.kvh = x % n_kv;
    x /= n_kv;
    const int s_splits = a.splits - a.p_splits;
    w.split = x % s_splits;
    w.tile = x / s_splits;
    w.per = a.split_blocks;
    w.slot = a.p_splits + w.split;
  }
  return w;
}

// Length of a group's prefix, within its table row.
__device__ __forceinline__ int prefix_of(const AttnArgs &a, int g) {
  return min(max(a.prefix_len[g], 0), a.b.cols << a.kv.page_shift);
}
__device__ __forceinline__ int group_at(const AttnArgs &a, int g) { return min(max(a.group_start[g], 0), a.b.n_seqs); }

// The x-th row tile of the prefixes.  Group g's tiles start at floor(first token G / rows) + g.
__device__ __forceinline__ bool find_prefix_tile(const AttnArgs &a, int x, Tile &t) {
  const Batch &b = a.b;
  const int g = wave_find(a.n_groups, x, [&](int i) { return (int64_t)b.q_start[group_at(a, i)] * a.G / kAttnTile + i; });
  const int s0 = group_at(a, g), s1 = group_at(a, g + 1);
  Seq q;
  q.t0 = b.q_start[s0];
  const int t1 = b.q_start[s1];
  q.row = s0 < b.n_seqs ? batch_row(b, s0) : -1;
  q.n = q.t0 < 0 || t1 > a.T || s1 <= s0 ? 0 : max(t1 - q.t0, 0);
  t.t0 = q.t0;
  t.n = q.n;
  const int64_t r0 = ((int64_t)x - ((int64_t)q.t0 * a.G / kAttnTile + g)) * kAttnTile;
  if (r0 < 0 || r0 >= (int64_t)t.n * a.G) return false;
  t.r0 = (int)r0;
  t.nr = min(kAttnTile, t.n * a.G - t.r0);
  t.row = q.row;
  t.full = true;
  t.len = t.row < 0 ? 0 : prefix_of(a, g);
  t.first = t.len;
  t.lo = 0;
  t.hi = t.len;
  return true;
}

// Keys from the end of its group's prefix on: of a suffix's tile.
__device__ __forceinline__ void cut_prefix(const AttnArgs &a, int seq, Tile &t) {
  const int g = wave_find(a.n_groups, seq, [&](int i) { return (int64_t)a.group_start[i]; });
  t.lo = min(prefix_of(a, g), t.hi);
}

// Values that not all rows of a tile see must be finite, for a hidden key's weight is 0: absent
// keys' values become zeros, and so do infinities and NaN.  Returns whether there were any.
template <bool F16>
__device__ __forceinline__ uint32_t make_finite(u32x4 &v, bool absent) {
  constexpr uint32_t m = F16 ? 0x7c007c00u : 0x7f807f80u;
  uint32_t bad = 0;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    // a half of t is 0 where its exponent is all ones, and otherwise at least 0x80, so taking 1
    // from it turns its top bit on in the first case only
    const uint32_t t = (v[j] & m) ^ m, z = ((t - 0x00010001u) & ~t & 0x80008000u) >> 15;
    v[j] &= absent ? 0u : ~(z * 0xffffu);
    bad |= z;
  }
  return absent ? 0u : bad;
}

// Adds the infinities and NaN that make_finite took out of blocks [b0, b1) to the results,
// already written, of the rows that see them: rows r0, r0 + step, ... below r1 (relative to the
// sequence).  part(r, token, head): where the row's partial results lie, or null: in out.
// Rare.  By a whole wave, for rows that no other wave writes.
template <int D, bool F16, class F>
__device__ void put_back(const AttnArgs &a, const Tile &t, int kvh, int b0, int b1, int all_lo, int all_hi, int r0,
                         int r1, int step, F part) {
  const int lane = threadIdx.x & 63;
  const TableRow trow = table_row(a, t.row);
  constexpr int kE = D / 64;
  for (int key = max(t.lo, b0 * kAttnKeys); key < min(t.hi, b1 * kAttnKeys); ++key) {
    const int k0 = key & ~(kAttnKeys - 1), page = page_at(a, trow, key);
    if ((k0 + kAttnKeys <= all_hi && k0 >= all_lo) || page < 0) continue;
    const uint16_t *v = a.kv.v + (int64_t)page * a.kv.ps + (int64_t)(key & ((1 << a.kv.page_shift) - 1)) * a.kv.ts +
                        (int64_t)kvh * a.kv.hs;
    float x[kE];
    bool any = false;
#pragma unroll
    for (int e = 0; e < kE; ++e) {
      const uint16_t w = v[lane * kE + e];
      x[e] = nonfinite16<F16>(w) ? unpack<F16>(w, false) : 0.0f;
      any |= nonfinite16<F16>(w);
    }
    if (!__ballot(any)) continue;
    for (int r = r0; r < r1; r += step) {
      const int64_t p = t.first + r / a.G;
      if ((!t.full && key > p) || (a.window && key <= p - a.window)) continue;
      const int64_t tk = t.t0 + r / a.G, hd = kvh * a.G + r % a.G;
      float *d = part(r, tk, hd);
#pragma unroll
      for (int e = 0; e < kE; ++e) {
        if (x[e] == 0.0f) continue;
        if (!d) {
          uint16_t *o = a.out.p + tk * a.out.ts + hd * a.out.hs + lane * kE + e;
          *o = (uint16_t)pack2<F16>(unpack<F16>(*o, false) + x[e], 0.0f);
        } else {
          d[lane * kE + e] += x[e];
        }
      }
    }
  }
}

template <int D>
struct Rows {
  static constexpr int kBuf = kAttnKeys * D * 2;         // V buffer of a wave, bytes
  static constexpr int kOStride = D + 4;                 // floats; padded against bank conflicts
  static constexpr int kOut = kAttnRows * kOStride * 4;  // a wave's partial output, over its buffer
  static constexpr int kWaveLds = kBuf > kOut ? kBuf : kOut;
  static constexpr int kLds = kWaves * kWaveLds;
};

// How k_attn_rows divides its work.  A segment is one (tile, key/value head); a sequence's
// segments have as many blocks of keys each as the longest of them, at least 1.  The blocks of
// all segments, one after the other, are cut into equal runs, one for each workgroup, so
// the lengths of the sequences do not matter.
struct SeqSize {
  int tiles, blocks;
};
__device__ __forceinline__ SeqSize seq_size(const AttnArgs &a, const Seq &q) {
  SeqSize z;
  z.tiles = (int)(((int64_t)q.n * a.G + kAttnRows - 1) / kAttnRows);
  const int len = min(max(q.total, 0), a.b.cols << a.kv.page_shift);
  const int64_t lo = a.window ? max((int64_t)q.total - q.n - a.window + 1, (int64_t)0) : 0;
  z.blocks = max(1, (int)((len + kAttnKeys - 1) / kAttnKeys - min(lo, (int64_t)len) / kAttnKeys));
  return z;
}
__device__ __forceinline__ int64_t total_blocks(const AttnArgs &a, const SeqSize &z) {
  return (int64_t)z.tiles * a.kv.n_kv * z.blocks;
}

__device__ __forceinline__ uint64_t div_u64(uint64_t x, uint64_t y) {
  return (x | y) >> 32 ? x / y : (uint32_t)x / (uint32_t)y;
}

// Runs of `total` blocks over `n` workgroups: the first `more` take one more than `each`.
struct Runs {
  int64_t each, more;
  int n;
  __device__ __forceinline__ Runs(int64_t total, int wgs) {
    const int64_t least = (total + kWaves - 1) / kWaves;  // a block for every wave
    n = (int)max(min((int64_t)wgs, least), (int64_t)1);
    each = (int64_t)div_u64((uint64_t)total, (uint64_t)n);
    more = total - each * n;
  }
  __device__ __forceinline__ int64_t start(int64_t w) const { return each * w + min(w, more); }
  __device__ __forceinline__ int holder(int64_t x) const {  // of block x
    const int64_t edge = more * (each + 1);
    return (int)(x < edge ? div_u64((uint64_t)x, (uint64_t)(each + 1)) : more + div_u64((uint64_t)(x - edge), (uint64_t)each));
  }
};

// Inclusive prefix sums over the wave's lanes, of numbers below 2^53: as binary64, whose DPP
// steps need no LDS.
__device__ __forceinline__ int64_t wave_incl_scan64(int64_t x) {
  double v = (double)x;
  v += dpp_d<0x111>(v);       // row_shr:1 (lanes without a source take 0)
  v += dpp_d<0x112>(v);       // row_shr:2
  v += dpp_d<0x114>(v);       // row_shr:4
  v += dpp_d<0x118>(v);       // row_shr:8
  v += dpp_d<0x142, 0xa>(v);  // row_bcast:15 into rows 1 and 3
  v += dpp_d<0x143, 0xc>(v);  // row_bcast:31 into rows 2 and 3
  return (int64_t)v;
}
__device__ __forceinline__ int64_t readlane64(int64_t x, int l) {
  return ((int64_t)__builtin_amdgcn_readlane((int)(x >> 32), l) << 32) | (uint32_t)__builtin_amdgcn_readlane((int)x, l);
}

// Walks the sequences from the one that holds a block on.  Up to 64 sequences are read once,
// one a lane; more of them are summed first and then searched 64 at a time.  Every wave does
// the same.
struct Walk {
  int s0;       // sequences s0 .. s0 + 63 are in the lanes
  Seq mine;
  int64_t size;  // blocks of this lane's sequence
  int at;       // lane of the current one
  int64_t cum;  // blocks before it

  __device__ __forceinline__ void read(const AttnArgs &a, int from) {
    s0 = from;
    const int s = from + (threadIdx.x & 63);
    mine = read_seq(a, min(s, a.b.n_seqs - 1));
    size = s < a.b.n_seqs ? total_blocks(a, seq_size(a, mine)) : 0;
  }
  // blocks of all sequences; leaves the first 64 in the lanes
  __device__ __forceinline__ int64_t total(const AttnArgs &a) {
    int64_t sum = 0;
    for (int s = (a.b.n_seqs - 1) / 64 * 64; s >= 0; s -= 64) {
      read(a, s);
      sum += readlane64(wave_incl_scan64(size), 63);
    }
    return sum;
  }
  // to the sequence that holds block x (below the total)
  __device__ __forceinline__ void find(const AttnArgs &a, int64_t x) {
    int64_t before = 0;
    while (true) {
      const int64_t inc = wave_incl_scan64(size), all = readlane64(inc, 63);
      if (x < before + all || s0 + 64 >= a.b.n_seqs) {
        const uint64_t over = __ballot(before + inc > x);
        at = over ? __builtin_ctzll(over) : 63;
        cum = before + readlane64(inc - size, at);
        return;
      }
      before += all;
      read(a, s0 + 64);
    }
  }
  // to the next sequence that has blocks (there is one)
  __device__ __forceinline__ void next(const AttnArgs &a) {
    cum += readlane64(size, at);
    uint64_t some = __ballot(size > 0) & ~((uint64_t(2) << at) - 1);
    while (!some && s0 + 64 < a.b.n_seqs) {
      read(a, s0 + 64);
      some = __ballot(size > 0);
    }
    at = some ? __builtin_ctzll(some) : 63;
  }
  __device__ __forceinline__ Seq seq() const { return readlane_seq(mine, at); }
};

// 16 rows against runs of blocks.  The four waves take blocks in turn; each holds the next block in
// registers while it works on one -- K as the matrix operand itself, V on its way to the wave's
// LDS buffer, from where it is read transposed.  (Blocks by direct-to-LDS loads and splits of
// fixed length took 203 us for the 64 sequences up to 16K that take 172 us here: long
// sequences kept a few compute units busy.)
template <int D, bool F16>
__global__ void __launch_bounds__(kThreads, D == 256 ? 1 : 2) k_attn_rows(AttnArgs a) {
  using L = Rows<D>;
  extern __shared__ __align__(16) uint8_t lds_raw[];
  __shared__ Stats ml[kWaves][kAttnRows];
  __shared__ int odd;  // some value that not all rows see is an infinity or NaN
  const int wg = blockIdx.x;
  const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63;

  // this workgroup's run, and the sequence where it starts
  Walk walk;
  const int64_t total = walk.total(a);
  const Runs runs(total, a.wgs);
  if (tid == 0) {
    odd = 0;
    a.rec[wg].n = 0;  // results to be joined from this workgroup on: none so far
  }
  if (total == 0 || wg >= runs.n) return;
  int64_t cur = runs.start(wg);
  const int64_t end = runs.start(wg + 1);
  walk.find(a, cur);
  __syncthreads();

  const int n = lane & 15, g = lane >> 4;  // query row of the lane, lane group
  const uint32_t vbuf = lds_addr(lds_raw) + wave * L::kWaveLds;
  while (true) {
    const Seq sq = walk.seq();
    const SeqSize z = seq_size(a, sq);
    const int64_t cum = walk.cum;
    const int seg = (int)div_u64((uint64_t)(cur - cum), (uint64_t)z.blocks), o0 = (int)(cur - cum - (int64_t)seg * z.blocks);
    const int o1 = (int)min((int64_t)z.blocks, o0 + (end - cur));
    const int kvh = __builtin_amdgcn_readfirstlane(seg % a.kv.n_kv);
    Tile t;
    set_tile(a, sq, (int64_t)(seg / a.kv.n_kv) * kAttnRows, kAttnRows, t);

    // this lane's query row
    const int rr = t.r0 + n;
    const bool live = n < t.nr;
    const int tok = t.t0 + rr / a.G, head = kvh * a.G + rr % a.G;
    const int64_t pos = live ? t.first + rr / a.G : -1;
    // visible keys: first_key .. last_key
    const int last_key = (int)(a.full ? (live ? (int64_t)t.len - 1 : -1) : min(pos, (int64_t)t.len - 1));
    const int first_key = a.window ? (int)max(pos - a.window + 1, (int64_t)0) : 0;
    // every row of the tile sees all keys of [all_lo, all_hi); lanes without a row (queries of
    // zeros) go along, and nothing of theirs is stored
    const int64_t pf = t.first + t.r0 / a.G, pl = t.first + (t.r0 + t.nr - 1) / a.G;
    const int all_hi = (int)(a.full ? (int64_t)t.len : min(pf + 1, (int64_t)t.len));
    const int64_t all_lo = a.window ? pl - a.window + 1 : 0;

    // (lanes without a row read the tile's first one, and take zeros)
    const uint16_t *qp = a.q.p + (int64_t)(live ? tok : t.t0 + t.r0 / a.G) * a.q.ts +
                         (int64_t)(live ? head : kvh * a.G + t.r0 % a.G) * a.q.hs;
    u32x4 qf[D / 32];
#pragma unroll
    for (int c = 0; c < D / 32; ++c) qf[c] = *(const u32x4 *)(qp + 32 * c + 8 * g);
#pragma unroll
    for (int c = 0; c < D / 32; ++c)
      if (!live) qf[c] = u32x4{0, 0, 0, 0};

    // this run's blocks of the segment
    const int blk0 = t.lo / kAttnKeys, nblk = (t.hi + kAttnKeys - 1) / kAttnKeys - blk0;
    const int b0 = blk0 + min(nblk, o0), b1 = blk0 + min(nblk, o1);
    const bool alone = o0 == 0 && o1 == z.blocks;
    // partial results: of a segment that goes on in the next run, and of one from the run before
    const int64_t slot = (2 * (int64_t)wg + (o0 == 0)) * kAttnRows;

    f32x4 acc[D / 16];
#pragma unroll
    for (int d = 0; d < D / 16; ++d) acc[d] = f32x4{0, 0, 0, 0};
    float m = -INFINITY, l = 0.0f, es = 0.0f;

    const TableRow trow = table_row(a, t.row);
    const int pmask = (1 << a.kv.page_shift) - 1;
    auto page_of = [&](int key) { return page_at(a, trow, key); };
    auto base = [&](const uint16_t *plane, int page, int key) {
      return (const char *)uniform_ptr(plane + (int64_t)max(page, 0) * a.kv.ps + (int64_t)(key & pmask) * a.kv.ts +
                                       (int64_t)kvh * a.kv.hs);
    };
    // K comes in the layout of the matrix operand (lane: key n of a half, 8 elements from 8 g of
    // each 32), V in rows of whole cache lines
    constexpr int kChunks = D / 8, kRowsPer = 64 / kChunks, kVLoads = kAttnKeys / kRowsPer;
    const int ts2 = (int)a.kv.ts * 2;
    const int koff = n * ts2 + 16 * g, vrow = lane / kChunks;
    const int voff = vrow * ts2 + lane % kChunks * 16;
    u32x4 kr[2][D / 32], vr[kVLoads];
    auto load = [&](int key0, int pg0, int pg1) {
      const char *k0 = base(a.kv.k, pg0, key0), *k1 = base(a.kv.k, pg1, key0 + 16);
      const char *v0 = base(a.kv.v, pg0, key0), *v1 = base(a.kv.v, pg1, key0 + 16);
#pragma unroll
      for (int c = 0; c < D / 32; ++c) kr[0][c] = *(const u32x4 *)(k0 + koff + 64 * c);
#pragma unroll
      for (int c = 0; c < D / 32; ++c) kr[1][c] = *(const u32x4 *)(k1 + koff + 64 * c);
#pragma unroll
      for (int i = 0; i < kVLoads; ++i)
        vr[i] = *(const u32x4 *)((i < kVLoads / 2 ? v0 : v1) + (voff + i % (kVLoads / 2) * kRowsPer * ts2));
    };

    int blk = b0 + wave;
    int pg0 = -1, pg1 = -1;
    if (blk < b1) {
      pg0 = page_of(blk * kAttnKeys);
      pg1 = page_of(blk * kAttnKeys + 16);
      load(blk * kAttnKeys, pg0, pg1);
    }
    for (; blk < b1; blk += kWaves) {
      const int key0 = blk * kAttnKeys;
      // (a block behind the last one is not loaded: its numbers are those of this one)
      const int next = blk + kWaves < b1 ? key0 + kWaves * kAttnKeys : key0;
      const int npg0 = page_of(next), npg1 = page_of(next + 16);
      // keys present in the halves (behind the sequence's end, or in a bad page: absent)
      const int have0 = pg0 < 0 ? 0 : max(0, min(16, t.len - key0));
      const int have1 = pg1 < 0 ? 0 : max(0, min(16, t.len - key0 - 16));

      f32x4 s[2] = {f32x4{0, 0, 0, 0}, f32x4{0, 0, 0, 0}};
#pragma unroll
      for (int c = 0; c < D / 32; ++c)
#pragma unroll
        for (int h = 0; h < 2; ++h) s[h] = mfma16<F16>(kr[h][c], qf[c], s[h]);

      const bool edge = key0 + kAttnKeys > all_hi || key0 < all_lo;
      const bool whole = have0 + have1 == kAttnKeys && !edge;
      if (!whole) {
        uint32_t bad = 0;
#pragma unroll
        for (int i = 0; i < kVLoads; ++i) {
          const int r = i * kRowsPer + vrow;
          const bool absent = (r & 15) >= (r < 16 ? have0 : have1);
          if (edge) bad |= make_finite<F16>(vr[i], absent);
          else if (absent) vr[i] = u32x4{0, 0, 0, 0};
        }
        if (bad) odd = 1;
      }
#pragma unroll
      for (int i = 0; i < kVLoads; ++i) {
        const int r = i * kRowsPer + vrow;
        *(__attribute__((address_space(3))) u32x4 *)(uintptr_t)(vbuf + r * D * 2 + (((lane % kChunks) ^ swz<D>(r)) * 16)) = vr[i];
      }
      if (blk + kWaves < b1) load(next, npg0, npg1);

      float p[8];
      float mx = -INFINITY;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        float x = s[i / 4][i % 4] * a.scale_log2;
        if (!whole) {
          const int o = 4 * g + i % 4, key = key0 + 16 * (i / 4) + o;
          if (o >= (i / 4 ? have1 : have0) || key > last_key || key < first_key) x = -INFINITY;
        }
        p[i] = x;
        mx = fmaxf(mx, x);
      }
      const float mn = fmaxf(m, groups_max(mx));
      const float mu = mn == -INFINITY ? 0.0f : mn;  // nothing seen yet: exp2(-inf - 0) = 0
      const float f = __builtin_amdgcn_exp2f(m - mu);
      m = mn;
      float ps = 0.0f;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        p[i] = __builtin_amdgcn_exp2f(F16 ? p[i] - mu + rows_bias(F16) : p[i] - mu);
        ps += p[i];
      }
      es = es * f + ps;
      if (__ballot(f != 1.0f)) {
#pragma unroll
        for (int d = 0; d < D / 16; ++d) acc[d] *= f;
      }
      const u32x4 pf4 = {pack2<F16>(p[0], p[1]), pack2<F16>(p[2], p[3]), pack2<F16>(p[4], p[5]), pack2<F16>(p[6], p[7])};
      float ls = 0.0f;  // (of the block by itself: two keys at a time vanish in a long row's sum)
#pragma unroll
      for (int i = 0; i < 4; ++i) ls = add2<F16>(pf4[i], ls);
      l = l * f + ls;

      {
        const int vk = 4 * g + (n >> 2);  // LDS row this lane addresses for the transposing reads
#pragma unroll
        for (int d = 0; d < D / 16; ++d) {
          const int c = 2 * d + ((n & 3) >> 1);
          const uint32_t o = (uint32_t)((c ^ swz<D>(vk)) * 16 + (n & 1) * 8 + vk * D * 2);
          const uint32_t o2 = (uint32_t)((c ^ swz<D>(vk + 16)) * 16 + (n & 1) * 8 + (vk + 16) * D * 2);
          const uint64_t v0 = tr_read(vbuf + o), v1 = tr_read(vbuf + o2);
          const u32x4 vf = {(uint32_t)v0, (uint32_t)(v0 >> 32), (uint32_t)v1, (uint32_t)(v1 >> 32)};
          acc[d] = mfma16<F16>(vf, pf4, acc[d]);
        }
      }
      pg0 = npg0;
      pg1 = npg1;
    }

    // join the waves: each writes its rows over its own buffers
    l = groups_sum(l);
    es = groups_sum(es);
    float *o = (float *)(lds_raw + wave * L::kWaveLds);
#pragma unroll
    for (int d = 0; d < D / 16; ++d) *(f32x4 *)(o + n * L::kOStride + 16 * d + 4 * g) = acc[d];
    if (g == 0) {
      ml[wave][n] = Stats{m, l, es};
    }
    __syncthreads();
    constexpr int kVecs = D / 4;  // 4-element vectors of a row
    for (int i = tid; i < t.nr * kVecs; i += kThreads) {
      const int r = i / kVecs, c = (i % kVecs) * 4;
      float mw = ml[0][r].m;
#pragma unroll
      for (int w = 1; w < kWaves; ++w) mw = fmaxf(mw, ml[w][r].m);
      const float mu = mw == -INFINITY ? 0.0f : mw;
      f32x4 v = {0, 0, 0, 0};
      float sum = 0.0f, esum = 0.0f;
#pragma unroll
      for (int w = 0; w < kWaves; ++w) {
        const float f = __builtin_amdgcn_exp2f(ml[w][r].m - mu);
        sum += f * ml[w][r].l;
        esum += f * ml[w][r].e;
        v += f * *(const f32x4 *)((const float *)(lds_raw + w * L::kWaveLds) + r * L::kOStride + c);
      }
      const int q = t.r0 + r;
      const int64_t tk = t.t0 + q / a.G, hd = kvh * a.G + q % a.G;
      if (alone) {
        const float inv = reciprocal_of(sum);
        const uint2 w = {pack2<F16>(v[0] * inv, v[1] * inv), pack2<F16>(v[2] * inv, v[3] * inv)};
        *(uint2 *)(a.out.p + tk * a.out.ts + hd * a.out.hs + c) = w;
        if (a.lse && c == 0) a.lse[tk * a.H + hd] = lse_of(mw, esum, rows_bias(F16));
      } else {
        const int64_t at = slot + r;
        *(f32x4 *)(a.part + at * D + c) = v;
        if (c == 0) a.stats[at] = AttnStats{mw, sum, esum, 0.0f};
      }
    }
    if (odd) {  // (a barrier lies behind its last write)
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "agent");
      __syncthreads();
      put_back<D, F16>(a, t, kvh, b0, b1, (int)min(all_lo, (int64_t)INT32_MAX), all_hi, t.r0 + wave, t.r0 + t.nr, kWaves,
                       [&](int r, int64_t, int64_t) { return alone ? nullptr : a.part + (slot + r - t.r0) * D; });
    }
    if (o0 == 0 && o1 < z.blocks) {  // the first of the workgroups that share the segment
      if (tid == 0) a.rec[wg] = AttnRec{runs.holder(cum + (int64_t)(seg + 1) * z.blocks - 1) - wg + 1, t.t0, t.r0, t.nr, kvh};
      return;
    }
    cur += o1 - o0;
    if (cur == end) return;
    __syncthreads();  // buffers, sums and the flag are free again
    if (tid == 0) odd = 0;
    if (cur == cum + total_blocks(a, z)) walk.next(a);
    __syncthreads();
  }
}

// ---------------------------------------------------------------- tiles of many rows

__device__ __forceinline__ float halves_max(float v) {
  auto a = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return fmaxf(__uint_as_float(a[0]), __uint_as_float(a[1]));
}
__device__ __forceinline__ float halves_sum(float v) {
  auto a = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return __uint_as_float(a[0]) + __uint_as_float(a[1]);
}

__device__ __forceinline__ float uniform_f(float v) {
  return __int_as_float(__builtin_amdgcn_readfirstlane(__float_as_int(v)));
}

template <bool F16>
__device__ __forceinline__ f32x16 mfma32(u32x4 a, u32x4 b, f32x16 c) {
  if constexpr (F16)
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}

// N instructions of 64 chunks of 16 bytes from base on, to consecutive places of LDS.
template <int N>
__device__ __forceinline__ void dma_rows(const void *base, const uint32_t (&voff)[N], uint32_t lds) {
  const void *b = uniform_ptr(base);
  const uint32_t at = __builtin_amdgcn_readfirstlane(lds);
#define MOE_NEXT "s_add_u32 m0, m0, 0x400\n\ts_nop 0\n\t"
  if constexpr (N == 1)
    dma16(base, voff[0], lds);
  else if constexpr (N == 2)
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %3\n\t" MOE_NEXT
                 "global_load_lds_dwordx4 %2, %3\n" ::"s"(at), "v"(voff[0]), "v"(voff[1]), "s"(b)
                 : "memory", "m0", "scc");
  else
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %5\n\t" MOE_NEXT
                 "global_load_lds_dwordx4 %2, %5\n\t" MOE_NEXT "global_load_lds_dwordx4 %3, %5\n\t" MOE_NEXT
                 "global_load_lds_dwordx4 %4, %5\n" ::"s"(at), "v"(voff[0]), "v"(voff[1]), "v"(voff[2]), "v"(voff[3]), "s"(b)
                 : "memory", "m0", "scc");
#undef MOE_NEXT
}

__device__ __forceinline__ void lds_barrier() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// K and V blocks in LDS: one in use, the others in flight.  Two of 256-wide heads (64 KiB) leave
// room for two workgroups on a compute unit, whose matrix and vector phases then overlap: a
// 4096-token chunk at 32K takes 2042 us; three stages and one workgroup 3248 us, or 2073 us with
// eight waves.  Narrower heads have room for three.
constexpr int stages(int dim) { return dim == 256 ? 2 : 3; }

// A weight is 2^(s scale + fl(bias - m scale)), one fused operation, off by the rounding of the
// reference's term: below 2^-12 for scores (base-2 exponents) of up to 2^12, but from about 2^24 on by whole
// powers of two, and from 2^31 on every weight of a row is 0 or infinite.  Where a row's reference is
// further out than kFar, each of its scores is rounded as the reference is before the difference is
// taken, so that the largest weight is 1, and the reference does not lag.
constexpr float kFar = 4096.0f;
// What a wave is given the issue slots for while others of its SIMD do the other thing.  Measured
// with Matrix / Softmax / None: 4096 tokens at 32K, heads of 256, 1927 / 1997 / 2022 us; 4096 at
// 16K, heads of 128, 1150 / 1133 / 1101; 4096 at 8K, heads of 64, 211 / 199 / 216.
enum class First { Matrix, Softmax, None };

// 32 rows a wave, four waves.  A workgroup's waves pass one barrier a block: behind it the block is
// there for all, and the buffer of the block before it is free for the loads of the next.
// Waves on a SIMD: two, three, four by width (of 128, with 169 registers and so two waves, 24 ragged
// chunks take 143 us; with 168 and three, 132).
// PREFIX: of shared prefixes and the suffixes behind them (work_of); every result is partial.
template <int D, bool F16, bool PREFIX>
__global__ void __launch_bounds__(kThreads, D == 256 ? 2 : D == 128 ? 3 : 4) k_attn_tile(AttnArgs a) {
  constexpr int kBuf = kAttnKeys * D * 2;      // one K or V block, bytes
  constexpr int kStages = stages(D);
  constexpr First kFirst = D == 256 ? First::Matrix : D == 64 ? First::Softmax : First::None;
  constexpr int kInstr = kBuf / 1024 / kWaves;     // load instructions a wave issues for one block
  constexpr int kRowsPer = 512 / D;            // LDS rows of one instruction
  static_assert(kInstr == 1 || kInstr == 2 || kInstr == 4, "as dma_rows has them");
  extern __shared__ __align__(16) uint8_t lds_raw[];
  Tile t;
  // the key/value heads of one tile next to each other: 4096 tokens at 16K, 8 such heads of 128,
  // 1052 us; head after head 1128
  Work work{};
  if constexpr (PREFIX) {
    work = work_of(a, blockIdx.x);
  } else {
    work.tile = blockIdx.x / (unsigned)a.kv.n_kv;
    work.kvh = blockIdx.x - work.tile * a.kv.n_kv;
    work.split = work.slot = blockIdx.y;
    work.per = a.split_blocks;
  }
  const int kvh = work.kvh;
  int seq;
  if (PREFIX && work.prefix) {
    if (!find_prefix_tile(a, work.tile, t)) return;
  } else {
    if (!find_tile(a, work.tile, kAttnTile, t, seq)) return;
    if constexpr (PREFIX) cut_prefix(a, seq, t);
  }
  const bool full = PREFIX ? t.full : a.full;
  const int splits = !PREFIX ? a.splits : work.prefix ? a.p_splits : a.splits - a.p_splits;
  // Behind the buffers, so that these start at LDS address 0 (addresses are combined by
  // exclusive or): whether some value that not all rows see is an infinity or NaN.
  int &odd = *(int *)(lds_raw + kStages * 2 * kBuf);
  const int split = work.split;
  const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63;
  if (tid == 0) odd = 0;
  __syncthreads();
  const int n = lane & 31, half = lane >> 5;
  const uint32_t lds0 = lds_addr(lds_raw);

  // this lane's query row, and its wave's
  const int w0 = t.r0 + wave * 32;                               // first row of the wave
  const int wn = max(0, min(32, t.r0 + t.nr - w0));              // rows of the wave
  const int rr = w0 + n;
  const bool live = n < wn;
  const int tok = t.t0 + rr / a.G, head = kvh * a.G + rr % a.G;
  const int64_t pos = live ? t.first + rr / a.G : -1;
  const int last_key = (int)(full ? (live ? (int64_t)t.len - 1 : -1) : min(pos, (int64_t)t.len - 1));
  const int first_key = PREFIX ? t.lo : a.window ? (int)max(pos - a.window + 1, (int64_t)0) : 0;
  const int64_t pf = t.first + w0 / a.G, pl = t.first + (w0 + max(wn, 1) - 1) / a.G;
  // all rows of the wave see the keys of [all_lo, all_hi); some row sees those of [any_lo, any_hi)
  const int all_hi = (int)(full ? (int64_t)t.len : min(pf + 1, (int64_t)t.len));
  const int all_lo = PREFIX ? t.lo : a.window ? (int)max(pl - a.window + 1, (int64_t)0) : 0;
  const int any_hi = wn == 0 ? 0 : (int)(full ? (int64_t)t.len : min(pl + 1, (int64_t)t.len));
  const int any_lo = PREFIX ? t.lo : a.window ? (int)max(pf - a.window + 1, (int64_t)0) : 0;

  // keys below all_lo_t and from all_hi_t on are hidden from some row of the tile
  const int64_t tf = t.first + t.r0 / a.G, tl = t.first + (t.r0 + t.nr - 1) / a.G;
  const int all_hi_t = (int)(full ? (int64_t)t.len : max(min(tf + 1, (int64_t)t.len), (int64_t)0));
  const int all_lo_t = PREFIX ? t.lo : a.window ? (int)max(tl - a.window + 1, (int64_t)0) : 0;

  const int blk0 = t.lo / kAttnKeys, nblk = (t.hi + kAttnKeys - 1) / kAttnKeys - blk0;
  const int b0 = blk0 + min(nblk, split * work.per);
  const int b1 = blk0 + (split + 1 == splits ? nblk : min(nblk, (split + 1) * work.per));

  // the rows that this wave loads lie in one 16-key half of a block
  const int my_r0 = wave * kInstr * kRowsPer, upper = my_r0 >> 4;
  // Pages are looked up 64 halves at a time, one a lane, and a block's read from the lanes (numbers
  // fetched and checked block by block take twice the scalar instructions: 4096 tokens at 32K 1898 us,
  // 1849 this way; one token at 500 11.6 and 11.2).
  constexpr int kPageStep = 16;  // blocks after which the next 64 halves are taken, which half overlap
  const int32_t *table = a.b.table + (int64_t)max(t.row, 0) * a.b.cols;
  auto pages_from = [&](int blk) {  // lane i: page of half i of the blocks from blk on, or -1
    const int col = (blk * kAttnKeys + lane * 16) >> a.kv.page_shift;
    const int page = table[min(col, a.b.cols - 1)];
    return col < a.b.cols && (unsigned)page < (unsigned)a.kv.n_pages ? page : -1;
  };
  // (asked for before the queries, whose arrival they need not wait for: one token at 4096 keys, 2 heads of 256,
  // 12.0 us and 12.6 otherwise; 24 ragged chunks, heads of 128, 125 and 129)
  int pages = pages_from(b0), more = b0 + kPageStep < b1 ? pages_from(b0 + kPageStep) : -1, from = b0;
  // a negative scale is taken as a positive one on negated queries, so that the largest score
  // is the largest product
  const float scale = a.scale_log2 == 0.0f ? 1.0f : fabsf(a.scale_log2);  // 0: of queries of zeros
  const uint32_t flip = a.scale_log2 < 0.0f ? 0x80008000u : 0u;
  // (lag: finite, so that it is exceeded from -infinity on)
  constexpr float kLag = lag_of(F16), kBias = tile_bias(F16);
  const float lag = uniform_f(fminf(kLag / scale, 1e30f)), far = uniform_f(lag * (kFar / kLag));
  // (lanes without a row read the tile's first one, and take zeros)
  const uint16_t *qp = a.q.p + (int64_t)(live ? tok : t.t0 + t.r0 / a.G) * a.q.ts +
                       (int64_t)(live ? head : kvh * a.G + t.r0 % a.G) * a.q.hs;
  u32x4 qf[D / 16];
#pragma unroll
  for (int c = 0; c < D / 16; ++c) qf[c] = *(const u32x4 *)(qp + 16 * c + 8 * half);
#pragma unroll
  for (int c = 0; c < D / 16; ++c) {
    if (!live || a.scale_log2 == 0.0f) qf[c] = u32x4{0, 0, 0, 0};
    qf[c] ^= flip;
  }

  uint32_t voff[kInstr];
#pragma unroll
  for (int i = 0; i < kInstr; ++i) {
    const int r = my_r0 + i * kRowsPer + lane / (D / 8);
    voff[i] = (uint32_t)(((r & 15) * (int)a.kv.ts + (((lane % (D / 8)) ^ swz<D>(r)) * 8)) * 2);
  }
  const char *kbase = (const char *)uniform_ptr(a.kv.k + (int64_t)kvh * a.kv.hs);
  const uint64_t page_bytes = 2 * a.kv.ps;
  const uint32_t row_bytes = 2 * (uint32_t)a.kv.ts;
  const int64_t to_v = (const char *)a.kv.v - (const char *)a.kv.k;
  const uint32_t in_page = ((1u << a.kv.page_shift) - 1) & ~15u;
  auto load = [&](int blk, int page, int stage) {
    const uint32_t row = ((uint32_t)blk * kAttnKeys + upper * 16) & in_page;
    const char *k = kbase + ((uint32_t)page * page_bytes + row * row_bytes);
    const uint32_t at = lds0 + stage * 2 * kBuf + wave * kInstr * 1024;
    dma_rows<kInstr>(k, voff, at);
    dma_rows<kInstr>(k + to_v, voff, at + kBuf);
  };

  f32x16 acc[D / 32];
#pragma unroll
  for (int d = 0; d < D / 32; ++d)
#pragma unroll
    for (int i = 0; i < 16; ++i) acc[d][i] = 0.0f;
  float m = -INFINITY, l = 0.0f, es = 0.0f;  // m: of the unscaled products

  uint64_t absent = __ballot(pages < 0);
  auto page_of = [&](int blk) { return __builtin_amdgcn_readlane(pages, 2 * (blk - from) + upper); };
  pages = max(pages, 0);
  if (b0 < b1) load(b0, page_of(b0), 0);
  if (kStages > 2 && b0 + 1 < b1) load(b0 + 1, page_of(b0 + 1), 1);
  int stage = 0;
  for (int blk = b0; blk < b1; ++blk) {
    const int key0 = blk * kAttnKeys;
    const uint32_t kbuf = lds0 + stage * 2 * kBuf, vbuf = kbuf + kBuf;
    if (kStages > 2 && blk + 1 < b1) wait_vm<2 * kInstr>(); else wait_vm<0>();
    if (blk - from == kPageStep) {
      from = blk;
      absent = __ballot(more < 0);
      pages = max(more, 0);
      if (from + kPageStep < b1) more = pages_from(from + kPageStep);
    }
    const uint32_t gone = (uint32_t)(absent >> (2 * (blk - from))) & 3;  // halves in bad pages
    const bool mine_gone = gone >> upper & 1;
    // where some key is hidden from some row, its weight there is 0 and its value must be
    // finite: absent keys' values (behind the end, in a bad page) become zeros, and so do
    // infinities and NaN, which are put back at the end where they are seen
    if (mine_gone || key0 + kAttnKeys > all_hi_t || key0 < all_lo_t) {
#pragma unroll
      for (int i = 0; i < kInstr; ++i) {
        const int r = my_r0 + i * kRowsPer + lane / (D / 8);
        auto *w = (__attribute__((address_space(3))) u32x4 *)(uintptr_t)(vbuf + (wave * kInstr + i) * 1024 + lane * 16);
        u32x4 v = *w;
        if (make_finite<F16>(v, mine_gone || key0 + r >= t.len)) odd = 1;
        *w = v;
      }
    }
    wait_lds();
    lds_barrier();
    if (blk + kStages - 1 < b1) load(blk + kStages - 1, page_of(blk + kStages - 1), stage == 0 ? kStages - 1 : stage - 1);
    stage = stage + 1 == kStages ? 0 : stage + 1;
    if (key0 >= any_hi || key0 + kAttnKeys <= any_lo) continue;

    // the chunk's number enters the swizzled address by exclusive or: one register and one
    // operation a read, instead of a register for every chunk; the swizzle leaves bits from the
    // eighth on alone, so these are added (in the instruction: 1779 -> 1768 us)
    const uint32_t ka = kbuf + n * D * 2 + (half ^ swz<D>(n)) * 16;
    f32x16 s;
#pragma unroll
    for (int i = 0; i < 16; ++i) s[i] = 0.0f;
    // K from LDS kAhead matrix instructions before its use: left to itself the compiler reads
    // each operand right before the instruction and waits out the latency every time
    constexpr int kSteps = D / 16;
    constexpr int kAhead = D == 256 ? 3 : 4;
    u32x4 kf[kAhead];
    auto read_k = [&](int c) {
      return *(const __attribute__((address_space(3))) u32x4 *)(uintptr_t)((ka ^ (c % 8 * 32)) + c / 8 * 256);
    };
#pragma unroll
    for (int c = 0; c < kAhead; ++c) kf[c] = read_k(c);
    if (kFirst == First::Matrix) __builtin_amdgcn_s_setprio(1);
#pragma unroll
    for (int c = 0; c < kSteps; ++c) {
      __builtin_amdgcn_sched_barrier(0);
      s = mfma32<F16>(kf[c % kAhead], qf[c], s);
      if (c + kAhead < kSteps) kf[c % kAhead] = read_k(c + kAhead);
    }
    if (kFirst == First::Matrix) __builtin_amdgcn_s_setprio(0);
    if (kFirst == First::Softmax) __builtin_amdgcn_s_setprio(1);
    __builtin_amdgcn_sched_barrier(0);
    // the first of V, for after the softmax; rows kr, kr + 8, kr + 16, kr + 24 (swz(kr + 8) =
    // swz(kr) ^ swz(8), and 16 changes nothing)
    const int l16 = lane & 15, kr = 4 * half + (l16 >> 2);
    const uint32_t va = vbuf + kr * D * 2 + (((2 * ((lane >> 4) & 1) + ((l16 & 3) >> 1)) ^ swz<D>(kr)) * 16 + (l16 & 1) * 8);
    auto read_v = [&](int i) {  // operand i: 32 columns from 32 (i / 2), keys 16 (i % 2) ..
      const uint32_t a0 = va ^ (i / 2 % 4 * 64), a1 = a0 ^ (swz<D>(8) * 16);
      const int r = 16 * (i % 2), far = i / 8 * 256;
      const uint64_t v0 = tr_read(a0 + r * D * 2 + far), v1 = tr_read(a1 + (r + 8) * D * 2 + far);
      return u32x4{(uint32_t)v0, (uint32_t)(v0 >> 32), (uint32_t)v1, (uint32_t)(v1 >> 32)};
    };
    constexpr int kAheadV = D == 256 ? 2 : 4;
    u32x4 vf[kAheadV];
#pragma unroll
    for (int i = 0; i < kAheadV; ++i) vf[i] = read_v(i);
    __builtin_amdgcn_sched_barrier(0);
    if (key0 + kAttnKeys > all_hi || key0 < all_lo || gone) {
      const int have0 = gone & 1 ? 0 : max(0, min(16, t.len - key0));
      const int have1 = gone & 2 ? 0 : max(0, min(16, t.len - key0 - 16));
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const int k = 8 * (i / 4) + 4 * half + i % 4, key = key0 + k;
        if ((k & 15) >= (i < 8 ? have0 : have1) || key > last_key || key < first_key) s[i] = -INFINITY;
      }
    }
    float mx = s[0];
#pragma unroll
    for (int i = 1; i < 16; ++i) mx = fmaxf(mx, s[i]);
    // the reference m follows the maximum only where it lags by more than kLag (as a base-2
    // exponent), so weights stay below 2^(kLag + kBias) and the outputs are hardly ever rescaled;
    // the scores of rows far out are taken relative to it here (each product rounded by itself: not
    // fused)
    mx = halves_max(mx);
    if (__ballot(mx > (fabsf(m) > far ? -INFINITY : m + lag))) {
      const float mn = fmaxf(m, mx);
      const float ms = mn == -INFINITY ? 0.0f : mn * scale;
      const float f = __builtin_amdgcn_exp2f(m * scale - ms);
      m = mn;
      if (__ballot(fabsf(m) > far && m > -INFINITY)) {
#pragma unroll
        for (int i = 0; i < 16; ++i) s[i] = fabsf(m) > far ? s[i] * scale - ms : s[i];
      }
      l *= f;
      es *= f;
#pragma unroll
      for (int d = 0; d < D / 32; ++d) acc[d] *= f;
    }
    // (nothing seen yet, m = -infinity, is far out, too)
    const float off = fabsf(m) > far ? kBias : __builtin_fmaf(-m, scale, kBias), to_exp = fabsf(m) > far ? 1.0f : scale;
    float ps = 0.0f;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      s[i] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[i], to_exp, off));
      ps += s[i];
    }
    es += ps;
    u32x4 pf4[2];
    // the block's sum by itself: two keys at a time vanish in a long row's sum eight times sooner.  In
    // two chains: with one, 4096 tokens at 8K, heads of 64, take 211 us, 186 so (184 added one by one)
    float ls[2] = {0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      pf4[i / 4][i % 4] = pack2<F16>(s[2 * i], s[2 * i + 1]);
      ls[i / 4] = add2<F16>(pf4[i / 4][i % 4], ls[i / 4]);
    }
    l += ls[0] + ls[1];

    constexpr int kParts = D / 16;
    if (kFirst == First::Matrix) __builtin_amdgcn_s_setprio(1);
    if (kFirst == First::Softmax) __builtin_amdgcn_s_setprio(0);
#pragma unroll
    for (int i = 0; i < kParts; ++i) {
      __builtin_amdgcn_sched_barrier(0);
      acc[i / 2] = mfma32<F16>(vf[i % kAheadV], pf4[i % 2], acc[i / 2]);
      if (i + kAheadV < kParts) vf[i % kAheadV] = read_v(i + kAheadV);
    }
    if (kFirst == First::Matrix) __builtin_amdgcn_s_setprio(0);
    __builtin_amdgcn_sched_barrier(0);
  }

  l = halves_sum(l);
  es = halves_sum(es);
  __syncthreads();
  const bool fix = odd != 0;
  if (!live && !fix) return;
  const int64_t row = (int64_t)tok * a.H + head;
  // a tile whose keys are all in the first split needs no join: its other splits are empty, and
  // the first one's sum of -1 says that the row is done
  const bool direct = !PREFIX && (a.splits == 1 || nblk <= a.split_blocks);
  if (!live || (direct && split > 0)) {
  } else if (direct) {
    const float inv = reciprocal_of(l);
    uint16_t *o = a.out.p + (int64_t)tok * a.out.ts + (int64_t)head * a.out.hs + 4 * half;
#pragma unroll
    for (int d = 0; d < D / 32; ++d)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint2 w = {pack2<F16>(acc[d][4 * i] * inv, acc[d][4 * i + 1] * inv),
                         pack2<F16>(acc[d][4 * i + 2] * inv, acc[d][4 * i + 3] * inv)};
        *(uint2 *)(o + 32 * d + 8 * i) = w;
      }
    if (a.lse && half == 0) a.lse[row] = lse_of(m == -INFINITY ? m : m * scale, es, tile_bias(F16));
    if (a.splits > 1 && half == 0) a.stats[row * a.splits].l = -1.0f;
  } else {
    const int64_t at = row * a.splits + work.slot;
    if (b0 < b1) {
#pragma unroll
      for (int d = 0; d < D / 32; ++d)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          *(f32x4 *)(a.part + at * D + 32 * d + 8 * i + 4 * half) =
              f32x4{acc[d][4 * i], acc[d][4 * i + 1], acc[d][4 * i + 2], acc[d][4 * i + 3]};
    }
    if (half == 0) a.stats[at] = AttnStats{m == -INFINITY ? m : m * scale, l, es, 0.0f};
  }
  if (!fix) return;
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "agent");
  put_back<D, F16>(a, t, kvh, b0, b1, all_lo_t, all_hi_t, t.r0 + wave * 32, t.r0 + wave * 32 + wn, 1,
                   [&](int, int64_t tk, int64_t hd) {
                     return direct ? nullptr : a.part + ((tk * a.H + hd) * a.splits + work.slot) * D;
                   });
}

// Join the splits' partial results: one workgroup per (token, head).  Every wave holds the
// splits' weights, split s in lane s % 64; D / 4 threads take the splits of their group in
// turn, four loads in flight, and the groups' sums are added in LDS.  Splits without keys have
// weight 0 and their outputs are not read (they are not written either).  NT threads: 256 where
// their loads of one round reach all splits, 512 for more of them (one token at 4096 keys, 65
// splits, 12.1 us, 13.1 with 256; 16 sequences at 500, 9 splits, 12.0 with 256, 12.3 with 512).
constexpr int kJoinLoads = 4;
constexpr int one_round(int dim) { return kJoinLoads * kThreads / (dim / 4); }
template <int D, bool F16, int NT>
__global__ void __launch_bounds__(NT) k_attn_join(AttnArgs a) {
  constexpr int kVecs = D / 4, kGroups = NT / kVecs, kRegs = kMaxSplits / 64;
  __shared__ f32x4 sums[kGroups][kVecs];
  __shared__ float weight[kMaxSplits];
  const int64_t r = blockIdx.x;
  const int tid = threadIdx.x, lane = tid & 63;
  const int64_t tk = r / a.H, hd = r % a.H;
  if (tk >= a.b.q_start[a.b.n_seqs]) return;
  if (a.stats[r * a.splits].l < 0.0f) return;  // done already
  AttnStats st[kRegs];
  float mw = -INFINITY;
#pragma unroll
  for (int i = 0; i < kRegs; ++i) {
    st[i] = AttnStats{-INFINITY, 0.0f, 0.0f, 0.0f};
    if (64 * i + lane < a.splits) st[i] = a.stats[r * a.splits + 64 * i + lane];
    mw = fmaxf(mw, st[i].m);
  }
  mw = wave_max(mw);
  const float mu = mw == -INFINITY ? 0.0f : mw;
  float sum = 0.0f, esum = 0.0f;
#pragma unroll
  for (int i = 0; i < kRegs; ++i) {
    const float f = st[i].l == 0.0f ? 0.0f : __builtin_amdgcn_exp2f(st[i].m - mu);
    sum += f * st[i].l;
    esum += f * st[i].e;
    if (tid < 64) weight[64 * i + lane] = f;
  }
  sum = wave_sum(sum);
  esum = wave_sum(esum);
  __syncthreads();
  const int c = tid % kVecs, g = tid / kVecs;
  const f32x4 *p = (const f32x4 *)(a.part + r * a.splits * D) + c;
  f32x4 v = {0, 0, 0, 0};
  for (int s0 = g; s0 < a.splits; s0 += kJoinLoads * kGroups) {
    f32x4 x[kJoinLoads];
    float w[kJoinLoads];
#pragma unroll
    for (int i = 0; i < kJoinLoads; ++i) {
      const int s = s0 + i * kGroups;
      w[i] = s < a.splits ? weight[s] : 0.0f;
      x[i] = f32x4{0, 0, 0, 0};
      if (w[i] != 0.0f) x[i] = p[(int64_t)s * kVecs];
    }
#pragma unroll
    for (int i = 0; i < kJoinLoads; ++i) v += w[i] * x[i];
  }
  sums[g][c] = v;
  __syncthreads();
  if (g > 0) return;
#pragma unroll
  for (int i = 1; i < kGroups; ++i) v += sums[i][c];
  const float inv = reciprocal_of(sum);
  *(uint2 *)(a.out.p + tk * a.out.ts + hd * a.out.hs + 4 * c) =
      make_uint2(pack2<F16>(v[0] * inv, v[1] * inv), pack2<F16>(v[2] * inv, v[3] * inv));
  if (a.lse && tid == 0) a.lse[r] = lse_of(mw, esum, tile_bias(F16));
}

// The same for up to kFewSplits splits, where there are many rows: kRows rows a wave, their loads
// in flight together.  D / 4 lanes take a split, so 64 / (D / 4) of them are read at once and
// summed across lanes.
constexpr int kFewSplits = 4;
template <int D, bool F16>
__global__ void __launch_bounds__(kThreads) k_attn_join_few(AttnArgs a) {
  constexpr int kVecs = D / 4, kGroups = 64 / kVecs, kN = kFewSplits / kGroups, kRows = 4;
  const int lane = threadIdx.x & 63, c = lane % kVecs, g = lane / kVecs;
  const int64_t r0 = ((int64_t)blockIdx.x * kWaves + (threadIdx.x >> 6)) * kRows;
  const int64_t end = (int64_t)min(a.T, a.b.q_start[a.b.n_seqs]) * a.H;
  AttnStats st[kRows][kN];
  bool todo[kRows];
#pragma unroll
  for (int j = 0; j < kRows; ++j) {
    const AttnStats *p = a.stats + min(r0 + j, (int64_t)a.T * a.H - 1) * a.splits;
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      const int s = g + i * kGroups;
      st[j][i] = p[min(s, a.splits - 1)];
      if (s >= a.splits) st[j][i] = AttnStats{-INFINITY, 0.0f, 0.0f, 0.0f};
    }
  }
  f32x4 x[kRows][kN];
#pragma unroll
  for (int j = 0; j < kRows; ++j) {
    // (a first sum of -1: the row is done)
    todo[j] = r0 + j < end && !(__int_as_float(__builtin_amdgcn_readfirstlane(__float_as_int(st[j][0].l))) < 0.0f);
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      x[j][i] = f32x4{0, 0, 0, 0};
      if (todo[j] && st[j][i].l != 0.0f)  // (empty splits are not written)
        x[j][i] = *((const f32x4 *)(a.part + ((r0 + j) * a.splits + g + i * kGroups) * D) + c);
    }
  }
#pragma unroll
  for (int j = 0; j < kRows; ++j) {
    if (!todo[j]) continue;
    float mw = -INFINITY, sum = 0.0f, esum = 0.0f;
    f32x4 v = {0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < kN; ++i) mw = fmaxf(mw, st[j][i].m);
#pragma unroll
    for (int o = kVecs; o < 64; o <<= 1) mw = fmaxf(mw, __shfl_xor(mw, o, 64));
    const float mu = mw == -INFINITY ? 0.0f : mw;
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      const float f = __builtin_amdgcn_exp2f(st[j][i].m - mu);
      sum += f * st[j][i].l;
      esum += f * st[j][i].e;
      v += f * x[j][i];
    }
#pragma unroll
    for (int o = kVecs; o < 64; o <<= 1) {
      sum += __shfl_xor(sum, o, 64);
      esum += __shfl_xor(esum, o, 64);
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] += __shfl_xor(v[e], o, 64);
    }
    if (g > 0) continue;
    const int64_t r = r0 + j, tk = r / a.H, hd = r % a.H;
    const float inv = reciprocal_of(sum);
    *(uint2 *)(a.out.p + tk * a.out.ts + hd * a.out.hs + 4 * c) =
        make_uint2(pack2<F16>(v[0] * inv, v[1] * inv), pack2<F16>(v[2] * inv, v[3] * inv));
    if (a.lse && lane == 0) a.lse[r] = lse_of(mw, esum, tile_bias(F16));
  }
}

// Join the runs' partial results of segments that several workgroups share: workgroup x takes
// the segment, if any, that starts in run x, rows in turn.  Run x's results lie in its second
// slot, the following runs' in their first ones.
constexpr int kJoinThreads = 512;

template <int D, bool F16>
__global__ void __launch_bounds__(kJoinThreads) k_attn_join_runs(AttnArgs a) {
  constexpr int kVecs = D / 4, kGroups = kJoinThreads / kVecs, kW = kJoinThreads / 64;
  __shared__ f32x4 sums[kGroups][kVecs];
  __shared__ float weight[kMaxRuns], red[3][kW];
  const int wg = blockIdx.x;
  const AttnRec rec = a.rec[wg];
  const int tid = threadIdx.x, lane = tid & 63;
  const int c = tid % kVecs, g = tid / kVecs;
  for (int r = blockIdx.y; rec.n > 0 && r < rec.nr; r += gridDim.y) {
    auto at = [&](int s) { return (2 * (int64_t)(wg + s) + (s == 0)) * kAttnRows + r; };
    float mw = -INFINITY;
    for (int s = tid; s < rec.n; s += kJoinThreads) mw = fmaxf(mw, a.stats[at(s)].m);
    mw = wave_max(mw);
    if (lane == 0) red[0][tid >> 6] = mw;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kW; ++i) mw = fmaxf(mw, red[0][i]);
    const float mu = mw == -INFINITY ? 0.0f : mw;
    float sum = 0.0f, esum = 0.0f;
    for (int s = tid; s < rec.n; s += kJoinThreads) {
      const AttnStats st = a.stats[at(s)];
      const float f = __builtin_amdgcn_exp2f(st.m - mu);
      sum += f * st.l;
      esum += f * st.e;
      weight[s] = f;
    }
    sum = wave_sum(sum);
    esum = wave_sum(esum);
    if (lane == 0) {
      red[1][tid >> 6] = sum;
      red[2][tid >> 6] = esum;
    }
    __syncthreads();
    sum = esum = 0.0f;
#pragma unroll
    for (int i = 0; i < kW; ++i) {
      sum += red[1][i];
      esum += red[2][i];
    }
    f32x4 v = {0, 0, 0, 0};
    for (int s0 = g; s0 < rec.n; s0 += 8 * kGroups) {
      f32x4 x[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = *(const f32x4 *)(a.part + at(min(s0 + i * kGroups, rec.n - 1)) * D + 4 * c);
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (s0 + i * kGroups < rec.n) v += weight[s0 + i * kGroups] * x[i];
    }
    sums[g][c] = v;
    __syncthreads();
    if (g == 0) {
#pragma unroll
      for (int i = 1; i < kGroups; ++i) v += sums[i][c];
      const float inv = reciprocal_of(sum);
      const int64_t tk = rec.t0 + (rec.r0 + r) / a.G, hd = rec.kvh * a.G + (rec.r0 + r) % a.G;
      *(uint2 *)(a.out.p + tk * a.out.ts + hd * a.out.hs + 4 * c) =
          make_uint2(pack2<F16>(v[0] * inv, v[1] * inv), pack2<F16>(v[2] * inv, v[3] * inv));
      if (a.lse && tid == 0) a.lse[tk * a.H + hd] = lse_of(mw, esum, rows_bias(F16));
    }
    __syncthreads();
  }
}

// Joins a.splits partial results of every row.
template <int D, bool F16>
void join(const AttnArgs &a, hipStream_t s) {
  if (a.splits > one_round(D))
    hipLaunchKernelGGL((k_attn_join<D, F16, 512>), dim3(a.T * a.H), dim3(512), 0, s, a);
  else if (a.splits > kFewSplits)
    hipLaunchKernelGGL((k_attn_join<D, F16, kThreads>), dim3(a.T * a.H), dim3(kThreads), 0, s, a);
  else
    hipLaunchKernelGGL((k_attn_join_few<D, F16>), dim3(((int64_t)a.T * a.H + 4 * kWaves - 1) / (4 * kWaves)), dim3(kThreads), 0, s, a);
}

template <int D, bool F16>
hipError_t launch(const AttnArgs &a, hipStream_t s) {
  constexpr int lds = stages(D) * 2 * kAttnKeys * D * 2 + 16;
  if (a.n_groups > 0) {
    static std::atomic<uint64_t> done{0};
    const hipError_t e = allow_lds(k_attn_tile<D, F16, true>, lds, done);
    if (e != hipSuccess) return e;
    const int wgs = a.kv.n_kv * (a.p_tiles * a.p_splits + a.tiles * (a.splits - a.p_splits));
    hipLaunchKernelGGL((k_attn_tile<D, F16, true>), dim3(wgs), dim3(kThreads), lds, s, a);
    join<D, F16>(a, s);
  } else if (a.rows == kAttnRows) {
    static std::atomic<uint64_t> done{0};
    const hipError_t e = allow_lds(k_attn_rows<D, F16>, Rows<D>::kLds, done);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL((k_attn_rows<D, F16>), dim3(a.wgs), dim3(kThreads), Rows<D>::kLds, s, a);
    hipLaunchKernelGGL((k_attn_join_runs<D, F16>), dim3(a.wgs, a.join_rows), dim3(kJoinThreads), 0, s, a);
  } else {
    static std::atomic<uint64_t> done{0};
    const hipError_t e = allow_lds(k_attn_tile<D, F16, false>, lds, done);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL((k_attn_tile<D, F16, false>), dim3(a.tiles * a.kv.n_kv, a.splits), dim3(kThreads), lds, s, a);
    if (a.splits > 1) join<D, F16>(a, s);
  }
  return hipGetLastError();
}

}  // namespace

AttnShape attn_shape(int64_t T, int n_seqs, int64_t max_q, int64_t max_kv, int window, int H, int n_kv, int dim) {
  AttnShape s{};
  const int64_t G = H / n_kv;
  // Tiles of few rows over many long sequences: equal runs of keys (k_attn_rows).  Otherwise the
  // chunk kernel, its keys split: several workgroups on a compute unit hide each other's starts.
  // Measured on decodes of heads of 256 / 128 / 64, us with runs and with splits: 64 sequences up
  // to 16K 174 and 203; 64 up to 4K 104 and 142; 32 up to 8K 60 and 97; but one at 4K 16.1 and
  // 12.1, 16 up to 8K 39 and 30, 64 up to 1200 37 and 25, 200 up to 300 46 and 21.  More than
  // 16 rows a sequence: 16 sequences of 4 tokens and 8 heads at 8K 43 and 32.
  // A window bounds the keys, and makes the sequences that exceed it equally long, so that splits are
  // good up to twice as many: 64 sequences up to 16K (or 32K, heads of 256), windows of 128 keys and
  // of 16, 32 and 64 widths, heads of 256 29, 119, 210, 393 and 15, 108, 199, 382; of 128 30, 120,
  // 212, 397 and 15, 106, 200, 386; of 64 25, 66, 117, 209 and 15, 64, 118, 228; of lengths spread
  // evenly over their logarithm, heads of 256 28, 88, 120, 140 and 15, 69, 110, 192.
  if (window > 0 && max_kv > window + max_q) max_kv = window + max_q;
  const bool runs = max_q * G <= kAttnRows && (int64_t)n_seqs * n_kv >= 48 &&
                    max_kv >= (window > 0 ? 32 : 16) * (int64_t)dim;
  s.rows = runs ? kAttnRows : kAttnTile;
  s.tiles = (int)(T * G / s.rows + n_seqs);
  if (T == 0) return s;
  if (s.rows == kAttnRows) {
    s.splits = 1;
    s.wgs = runs_of(dim);
    s.join_rows = (int)(max_q * G < 1 ? 1 : max_q * G < kAttnRows ? max_q * G : kAttnRows);
    const size_t slots = (size_t)2 * s.wgs * kAttnRows;
    s.off_stats = slots * dim * 4;
    s.off_rec = s.off_stats + slots * sizeof(AttnStats);
    s.ws_bytes = s.off_rec + s.wgs * sizeof(AttnRec);
    return s;
  }
  // tiles that can hold rows, and splits that fill the chip with them
  int64_t busy = (max_q * G + s.rows - 1) / s.rows;
  busy = (busy < 1 ? 1 : busy) * n_seqs;
  if (busy < T * G / s.rows) busy = T * G / s.rows;  // (whatever max_q says)
  if (busy > s.tiles) busy = s.tiles;
  busy *= n_kv;
  const int64_t want = tile_slots(dim) / (busy < 1 ? 1 : busy);
  const int64_t blocks = (max_kv + kAttnKeys - 1) / kAttnKeys + 1;
  int64_t per = (blocks + (want < 1 ? 1 : want) - 1) / (want < 1 ? 1 : want);  // blocks of a split
  // Two blocks at least: one token at 4096 keys, 2 heads of 256, 12.1 us, 12.7 with one block (at 500
  // keys 11.1 and 10.3; four blocks took 2 us more there).  Few blocks are not split at all: 8 heads of
  // 128, 160 keys 8.9 us, 11.4 split; but 250 keys of 2 heads of 256 15.5 and 11.5.
  if (per < 2) per = 2;
  if (blocks <= kWhole) per = blocks;
  if (per * kMaxSplits < blocks) per = (blocks + kMaxSplits - 1) / kMaxSplits;
  s.splits = T * H > 1 << 22 ? 1 : (int)((blocks + per - 1) / per);
  s.split_blocks = (int)per;
  if (s.splits > 1) {
    const size_t rows = (size_t)T * H * s.splits;
    s.off_stats = (rows * dim * 4 + 255) & ~(size_t)255;
    s.ws_bytes = s.off_stats + rows * sizeof(AttnStats);
  }
  return s;
}

AttnShape prefix_shape(int64_t T, int n_seqs, int n_groups, int64_t max_q, int64_t max_prefix, int64_t max_suffix, int H, int n_kv,
                       int dim) {
  AttnShape s{};
  const int64_t G = H / n_kv;
  s.rows = kAttnTile;
  // (as find_prefix_tile and find_tile lay them out)
  s.p_tiles = (int)((T * G + kAttnTile - 1) / kAttnTile + n_groups - 1);
  s.tiles = (int)((T * G + kAttnTile - 1) / kAttnTile + n_seqs - 1);
  if (T == 0) return s;
  const int p_blocks = (int)((max_prefix + kAttnKeys - 1) / kAttnKeys), s_blocks = (int)((max_suffix + kAttnKeys - 1) / kAttnKeys) + 1;
  // tiles that can hold rows
  int64_t s_busy = (max_q * G + kAttnTile - 1) / kAttnTile;
  s_busy = (s_busy < 1 ? 1 : s_busy) * n_seqs;
  if (s_busy < T * G / kAttnTile) s_busy = T * G / kAttnTile;  // (whatever max_q says)
  if (s_busy > s.tiles) s_busy = s.tiles;
  int64_t p_busy = (T * G + kAttnTile - 1) / kAttnTile;
  if (p_busy < n_groups) p_busy = n_groups;
  // Blocks of a split, for prefixes and for suffixes: of some lengths those of least estimated time, in blocks (about
  // 0.95 us, heads of 256).  It is kFixed for the first workgroups' start, and the most of: the longest workgroup's, where
  // two whose rows are all there gain little from a compute unit in common; the work of all of them over
  // the compute units; and that of the workgroups in the order in which they find
  // place.  Then the join, which reads each split's results.  us so, and with the best pair of all lengths: 64
  // sequences of up to 512 keys behind 16384, 2 heads of 256, 41.7 and 40.3 (58.6 where splits just filled the chip);
  // 128 of them 59.6 both; 23 of 5 prefixes of up to 5000, drafts of up to 4 tokens, 32/8 heads of 128, 28.8 and 27.9; 64
  // of 64 prefixes of up to 2000 40 and 39; 64 of 2048, 32/8 heads of 128, 21.6 and 21.0; 64 of up to 512 behind 512
  // 25 and 22.  (Heads of 64, whose blocks are shorter while starts are not: 64 sequences of up to 512 keys behind 16384, 2
  // heads, 24.4; other lengths were not tried there.)
  constexpr double kFixed = 6.0, kNext = 1.5;  // (kNext: a further workgroup's start, while others run)
  constexpr int kUnits = 256;
  const int slots = (dim == 256 ? 2 : 3) * kUnits;
  const double join = 2e-6 * (double)(T * H) * dim;
  auto full = [&](int64_t busy) { return std::min(std::max((double)(T * G) / (double)(busy * kAttnTile), 0.25), 1.0); };
  const double p_full = full(p_busy), s_full = full(s_busy);
  auto splits = [](int blocks, int per) { return blocks > 0 ? (blocks + per - 1) / per : 1; };
  auto time = [&](int p_per, int s_per) {
    const int ps = splits(p_blocks, p_per), ss = splits(s_blocks, s_per);
    if (ps + ss > kMaxSplits) return 1e300;
    const int p_len = std::min(p_per, p_blocks), s_len = std::min(s_per, s_blocks);
    const int64_t p_all = p_busy * ps * n_kv, s_all = s_busy * ss * n_kv;
    const double longest = std::max(p_len * std::max(1.0, 1.2 * p_full * (double)((p_all + kUnits - 1) / kUnits)), (double)s_len);
    const double work = ((double)p_all * p_len * p_full + (double)s_all * s_len * s_full) * (1.0 / kUnits);
    // rounds of prefixes, suffixes in the places that the last of these leaves, and those that find none
    const double p_one = p_len + kNext, s_one = s_len + kNext;
    const int64_t p_rounds = (p_all + slots - 1) / slots, beside = (p_rounds * slots - p_all) * (int)(p_one / s_one);
    const double ends = (double)p_rounds * p_one - kNext + (s_all > beside ? (double)((s_all - beside + slots - 1) / slots) * s_one : 0.0);
    const double even = ((double)p_all * p_one + (double)s_all * s_one) / slots;  // (at least this, and not much more)
    const double places = std::max(even, std::min(ends, even + std::max(p_len, s_len)));
    return kFixed + std::max(std::max(longest, work), places) + join * (ps + ss);
  };
  // lengths: geometric ones, those that give each compute unit the same number of prefixes' workgroups, and the one that
  // leaves each suffix a place beside them
  const int most = p_blocks > s_blocks ? p_blocks : s_blocks;
  auto best_of = [&](auto t) {
    int best = 2;
    double least = 1e300;
    auto take = [&](int l) {
      const double v = t(l);
      if (v < least) least = v, best = l;
    };
    for (int l = 2; l <= most + l / 3; l += 1 + l / 4) take(l);
    for (int r = 0; r <= 3; ++r) {
      const int64_t ps = (r > 0 ? r * kUnits : slots - s_busy * n_kv) / (p_busy * n_kv);
      if (ps > 0 && p_blocks > 2 * ps) take((int)((p_blocks + ps - 1) / ps));
    }
    return best;
  };
  int p_per = best_of([&](int l) { return time(l, l); }), s_per = best_of([&](int l) { return time(p_per, l); });
  // (a launch holds less than 2^32 work-items; groups and sequences without tokens count)
  auto many = [&] { return n_kv * ((int64_t)s.p_tiles * splits(p_blocks, p_per) + (int64_t)s.tiles * splits(s_blocks, s_per)) >= int64_t(1) << 24; };
  while (splits(p_blocks, p_per) + splits(s_blocks, s_per) > kMaxSplits || many()) {
    p_per += 1 + p_per / 4;
    s_per += 1 + s_per / 4;
  }
  s.p_splits = splits(p_blocks, p_per);
  s.splits = s.p_splits + splits(s_blocks, s_per);
  s.p_blocks = p_per;
  s.split_blocks = s_per;
  const size_t rows = (size_t)T * H * s.splits;
  s.off_stats = (rows * dim * 4 + 255) & ~(size_t)255;
  s.ws_bytes = s.off_stats + rows * sizeof(AttnStats);
  return s;
}

hipError_t launch_paged_attn(const AttnArgs &a, hipStream_t s) {
  if (a.T <= 0) return hipSuccess;
  switch (a.kv.dim + (a.kv.fp16 ? 1 : 0)) {
    case 64: return launch<64, false>(a, s);
    case 65: return launch<64, true>(a, s);
    case 128: return launch<128, false>(a, s);
    case 129: return launch<128, true>(a, s);
    case 256: return launch<256, false>(a, s);
    case 257: return launch<256, true>(a, s);
  }
  return hipErrorInvalidValue;
}

}  // namespace moe
