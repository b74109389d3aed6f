// Attention of a ragged batch of new tokens over the paged cache.
//
// Per query row: out = sum_j p_j v_j / sum_j p_j, p_j = exp(scale q.k_j - m), with the running
// maximum m, sum and output rescaled as keys go by (one pass over K and V).  Scores, m, the
// sum and the output are binary32; p_j is rounded to the cache's type to enter the matrix
// units, and the sum is of the unrounded weights.
//
// k_attn_rows: a tile of 16 query rows -- (token, head) pairs of one key/value head, so the
// heads that share it share every load -- against one split of the keys.  Four waves take
// blocks of 32 keys in turn, each with a private 32-key K and V buffer in LDS filled by
// direct-to-LDS loads: the next block's K is in flight during softmax and P V, its V during
// the next Q K.  Both products are computed transposed with v_mfma_f32_16x16x32:
// S^T = K Q^T leaves a lane one query's scores, 4 keys at a time; with the contraction
// index of P V ordered the same way (slot j of lane group g is key 16 (j / 4) + 4 g + j % 4)
// those registers are P^T's operand as they are, and V^T comes from ds_read_b64_tr_b16.
// LDS rows are swizzled by 16-byte chunk so neither read has bank conflicts beyond its width.
// The waves' and then the splits' partial results are joined by their maxima, in fixed order.
//
// Bound: memory for single tokens (K and V read once per split).
#include <atomic>

#include "paged.hpp"

#pragma clang fp contract(off)

namespace moe {

namespace {

typedef __attribute__((__vector_size__(4 * sizeof(float)))) float f32x4;
typedef __attribute__((__vector_size__(8 * sizeof(_Float16)))) _Float16 f16x8;
typedef __attribute__((__vector_size__(4 * sizeof(short)))) short s16x4;

constexpr int kThreads = 256, kWaves = 4;
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
  if constexpr (F16)
    return (uint32_t)__builtin_bit_cast(uint16_t, (_Float16)lo) | (uint32_t)__builtin_bit_cast(uint16_t, (_Float16)hi) << 16;
  else
    return pack_bf16x2(lo, hi);
}
template <bool F16>
__device__ __forceinline__ float unpack(uint32_t w, bool hi) {
  const uint16_t v = (uint16_t)(hi ? w >> 16 : w & 0xffff);
  return F16 ? fp16_to_f32(v) : bf16_to_f32(v);
}
// whether a word of two values holds an infinity or NaN
template <bool F16>
__device__ __forceinline__ bool nonfinite(uint32_t w) {
  const uint32_t m = F16 ? 0x7c00u : 0x7f80u;
  return (w & m) == m || ((w >> 16) & m) == m;
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

// 16-byte chunk c of LDS row r lies at chunk c ^ swz(r): 16 rows at one chunk, and 16 rows of
// a 2-chunk column, then spread over all banks.
template <int D>
__device__ __forceinline__ int swz(int r) {
  return D == 64 ? (r >> 1) & 7 : r & 15;
}

// A tile's place in the batch: which sequence, its query rows and the keys they see.
struct Tile {
  int seq, row;       // row: of the table, -1: none
  int t0, n;          // first token, number of new tokens
  int r0, nr;         // first row (token * G + head) and rows of the tile
  int64_t first;      // position of the sequence's first new token
  int len;            // keys stored: min(kv_len, columns * page size)
  int lo, hi;         // keys that any row of the tile sees lie in [lo, hi)
};

// Tile x of `rows`-row tiles: sequence b's tiles start at floor(q_start[b] G / rows) + b,
// which leaves room for ceil(n_b G / rows) of them, so no list of tiles is needed.
__device__ __forceinline__ bool find_tile(const AttnArgs &a, int x, int rows, Tile &t) {
  const Batch &b = a.b;
  t.seq = wave_find(b.n_seqs, x, [&](int i) { return (int64_t)b.q_start[i] * a.G / rows + i; });
  t.t0 = b.q_start[t.seq];
  const int t1 = b.q_start[t.seq + 1];
  t.n = t1 - t.t0;
  if (t.t0 < 0 || t1 > a.T) return false;  // not a batch: touch nothing
  const int64_t r0 = ((int64_t)x - ((int64_t)t.t0 * a.G / rows + t.seq)) * rows;
  if (r0 < 0 || r0 >= (int64_t)t.n * a.G) return false;
  t.r0 = (int)r0;
  t.nr = min(rows, t.n * a.G - t.r0);
  t.row = batch_row(b, t.seq);
  const int total = t.row < 0 ? 0 : b.kv_len[t.row];
  t.first = (int64_t)total - t.n;
  t.len = min(max(total, 0), b.cols << a.kv.page_shift);
  const int64_t p0 = t.first + t.r0 / a.G, p1 = t.first + (t.r0 + t.nr - 1) / a.G;
  int64_t lo = 0, hi = t.len;
  if (!a.full && p1 + 1 < hi) hi = p1 + 1;
  if (a.window && p0 - a.window + 1 > lo) lo = p0 - a.window + 1;
  t.hi = (int)max(hi, (int64_t)0);
  t.lo = (int)min(lo, (int64_t)t.hi);
  return true;
}

template <int D>
struct Rows {
  static constexpr int kBuf = kAttnKeys * D * 2;         // one K or V buffer, bytes
  static constexpr int kWaveLds = 2 * kBuf;
  static constexpr int kOStride = D + 4;                 // floats; padded against bank conflicts
  static constexpr int kLds = kWaves * kWaveLds;
  static_assert(kAttnRows * kOStride * 4 <= kWaveLds, "a wave's partial output fits its buffers");
};

// 32 rows of one cache plane into LDS: keys key0 .. key0+31 lie in two 16-key halves of one
// page each.  The halves' bases are wave-uniform.
template <int D>
__device__ __forceinline__ void load_block(const uint16_t *h0, const uint16_t *h1, int64_t ts, uint32_t lds) {
  constexpr int kChunks = D / 8, kRowsPer = 64 / kChunks, kN = kAttnKeys / kRowsPer;
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int i = 0; i < kN; ++i) {
    const int r = i * kRowsPer + lane / kChunks;  // rows of one instruction lie in one half
    const int c = (lane % kChunks) ^ swz<D>(r);
    const uint32_t off = (uint32_t)(((r & 15) * (int)ts + c * 8) * 2);
    dma16(i < kN / 2 ? h0 : h1, off, lds + i * 1024);
  }
}

template <int D, bool F16>
__global__ void __launch_bounds__(kThreads, 1) k_attn_rows(AttnArgs a) {
  using L = Rows<D>;
  extern __shared__ __align__(16) uint8_t lds_raw[];
  __shared__ float ml[kWaves][2][kAttnRows];
  Tile t;
  if (!find_tile(a, blockIdx.x, kAttnRows, t)) return;
  const int kvh = blockIdx.y, split = blockIdx.z;
  const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63;
  const int n = lane & 15, g = lane >> 4;  // query row of the lane, lane group
  const uint32_t kbuf = lds_addr(lds_raw) + wave * L::kWaveLds, vbuf = kbuf + L::kBuf;

  // this lane's query row
  const int rr = t.r0 + n;
  const bool live = n < t.nr;
  const int tok = t.t0 + rr / a.G, head = kvh * a.G + rr % a.G;
  const int64_t pos = live ? t.first + rr / a.G : -1;
  // visible keys: first_key .. last_key
  const int last_key = (int)(a.full ? (live ? (int64_t)t.len - 1 : -1) : min(pos, (int64_t)t.len - 1));
  const int first_key = a.window ? (int)max(pos - a.window + 1, (int64_t)0) : 0;
  // every live row of the tile sees all keys of [all_lo, all_hi)
  const int64_t pf = t.first + t.r0 / a.G, pl = t.first + (t.r0 + t.nr - 1) / a.G;
  const int all_hi = (int)(a.full ? (int64_t)t.len : min(pf + 1, (int64_t)t.len));
  const int64_t all_lo = a.window ? pl - a.window + 1 : 0;

  u32x4 qf[D / 32];
#pragma unroll
  for (int c = 0; c < D / 32; ++c) {
    qf[c] = u32x4{0, 0, 0, 0};
    if (live) qf[c] = *(const u32x4 *)(a.q.p + (int64_t)tok * a.q.ts + (int64_t)head * a.q.hs + 32 * c + 8 * g);
  }

  // this split's blocks of 32 keys
  const int blk0 = t.lo / kAttnKeys, nblk = (t.hi + kAttnKeys - 1) / kAttnKeys - blk0;
  const int b0 = blk0 + (int)((int64_t)nblk * split / a.splits), b1 = blk0 + (int)((int64_t)nblk * (split + 1) / a.splits);

  f32x4 acc[D / 16];
#pragma unroll
  for (int d = 0; d < D / 16; ++d) acc[d] = f32x4{0, 0, 0, 0};
  float m = -INFINITY, l = 0.0f;

  // The page of the 16 keys from `key`, or -1; and its rows' base in one plane.
  const int32_t *trow = a.b.table + (int64_t)max(t.row, 0) * a.b.cols;
  const int pmask = (1 << a.kv.page_shift) - 1;
  auto page_of = [&](int key) {
    const int col = key >> a.kv.page_shift;
    const int page = col < a.b.cols ? trow[col] : -1;
    return __builtin_amdgcn_readfirstlane((unsigned)page < (unsigned)a.kv.n_pages ? page : -1);
  };
  auto base = [&](const uint16_t *plane, int page, int key) {
    return plane + (int64_t)max(page, 0) * a.kv.ps + (int64_t)(key & pmask) * a.kv.ts + (int64_t)kvh * a.kv.hs;
  };
  constexpr int kLoads = D / 16;  // load instructions of one block

  int blk = b0 + wave;
  int pg0 = -1, pg1 = -1;
  if (blk < b1) {
    pg0 = page_of(blk * kAttnKeys);
    pg1 = page_of(blk * kAttnKeys + 16);
    load_block<D>(base(a.kv.k, pg0, blk * kAttnKeys), base(a.kv.k, pg1, blk * kAttnKeys + 16), a.kv.ts, kbuf);
    load_block<D>(base(a.kv.v, pg0, blk * kAttnKeys), base(a.kv.v, pg1, blk * kAttnKeys + 16), a.kv.ts, vbuf);
  }
  for (; blk < b1; blk += kWaves) {
    const int key0 = blk * kAttnKeys;
    const bool more = blk + kWaves < b1;
    int npg0 = -1, npg1 = -1;
    if (more) {
      npg0 = page_of(key0 + kWaves * kAttnKeys);
      npg1 = page_of(key0 + kWaves * kAttnKeys + 16);
    }
    // keys present in the halves (behind the sequence's end, or in a bad page: absent)
    const int have0 = pg0 < 0 ? 0 : max(0, min(16, t.len - key0));
    const int have1 = pg1 < 0 ? 0 : max(0, min(16, t.len - key0 - 16));

    wait_vm<kLoads>();
    f32x4 s[2] = {f32x4{0, 0, 0, 0}, f32x4{0, 0, 0, 0}};
#pragma unroll
    for (int c = 0; c < D / 32; ++c)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int r = 16 * h + n;
        const u32x4 kf = *(const __attribute__((address_space(3))) u32x4 *)(uintptr_t)(kbuf + r * D * 2 +
                                                                                 (((4 * c + g) ^ swz<D>(r)) * 16));
        s[h] = mfma16<F16>(kf, qf[c], s[h]);
      }
    wait_lds();
    if (more)
      load_block<D>(base(a.kv.k, npg0, key0 + kWaves * kAttnKeys), base(a.kv.k, npg1, key0 + kWaves * kAttnKeys + 16),
                    a.kv.ts, kbuf);

    const bool whole = have0 + have1 == kAttnKeys && key0 + kAttnKeys <= all_hi && key0 >= all_lo && t.nr == kAttnRows;
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
      p[i] = __builtin_amdgcn_exp2f(p[i] - mu);
      ps += p[i];
    }
    l = l * f + ps;
    if (__ballot(f != 1.0f)) {
#pragma unroll
      for (int d = 0; d < D / 16; ++d) acc[d] *= f;
    }
    const u32x4 pf4 = {pack2<F16>(p[0], p[1]), pack2<F16>(p[2], p[3]), pack2<F16>(p[4], p[5]), pack2<F16>(p[6], p[7])};

    if (more) wait_vm<kLoads>(); else wait_vm<0>();
    bool odd = false;  // the block holds values that must not meet a zero weight
    if (!whole) {
      // absent keys' values become zeros; then look for infinities and NaN among the rest
      constexpr int kChunks = D / 8;
#pragma unroll
      for (int i = 0; i < kAttnKeys * kChunks / 64; ++i) {
        const int r = (i * 64 + lane) / kChunks;
        auto *w = (__attribute__((address_space(3))) u32x4 *)(uintptr_t)(vbuf + (i * 64 + lane) * 16);
        if ((r & 15) >= (r < 16 ? have0 : have1)) {
          *w = u32x4{0, 0, 0, 0};
        } else {
          const u32x4 v = *w;
          odd |= nonfinite<F16>(v[0]) || nonfinite<F16>(v[1]) || nonfinite<F16>(v[2]) || nonfinite<F16>(v[3]);
        }
      }
      odd = __ballot(odd) != 0;
      wait_lds();
    }
    if (!odd) {
      const int kr = 4 * g + (n >> 2);  // LDS row this lane addresses for the transposing reads
#pragma unroll
      for (int d = 0; d < D / 16; ++d) {
        const int c = 2 * d + ((n & 3) >> 1);
        const uint32_t o = (uint32_t)((c ^ swz<D>(kr)) * 16 + (n & 1) * 8 + kr * D * 2);
        const uint32_t o2 = (uint32_t)((c ^ swz<D>(kr + 16)) * 16 + (n & 1) * 8 + (kr + 16) * D * 2);
        const uint64_t v0 = tr_read(vbuf + o), v1 = tr_read(vbuf + o2);
        const u32x4 vf = {(uint32_t)v0, (uint32_t)(v0 >> 32), (uint32_t)v1, (uint32_t)(v1 >> 32)};
        acc[d] = mfma16<F16>(vf, pf4, acc[d]);
      }
    } else {
      // rare: values are summed key by key, for the rows that see the key only
      for (int k = 0; k < kAttnKeys; ++k) {
        const uint32_t w01 = (k & 2) ? pf4[k / 16 * 2 + 1] : pf4[k / 16 * 2];
        const float pk = unpack<F16>(__shfl(w01, n + 16 * ((k & 15) >> 2), 64), k & 1);
        const int key = key0 + k;
        const bool sees = (k & 15) < (k < 16 ? have0 : have1) && key <= last_key && key >= first_key;
#pragma unroll
        for (int d = 0; d < D / 16; ++d) {
          const int e = 16 * d + 4 * g;
          const uint64_t w = *(const __attribute__((address_space(3))) uint64_t *)(uintptr_t)(
              vbuf + k * D * 2 + (((e / 8) ^ swz<D>(k)) * 16 + (e & 4) * 2));
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float v = unpack<F16>((uint32_t)(i < 2 ? w : w >> 32), i & 1);
            acc[d][i] = sees ? __builtin_fmaf(pk, v, acc[d][i]) : acc[d][i];
          }
        }
      }
    }
    wait_lds();
    if (more)
      load_block<D>(base(a.kv.v, npg0, key0 + kWaves * kAttnKeys), base(a.kv.v, npg1, key0 + kWaves * kAttnKeys + 16),
                    a.kv.ts, vbuf);
    pg0 = npg0;
    pg1 = npg1;
  }

  // join the waves: each writes its rows over its own buffers
  l = groups_sum(l);
  float *o = (float *)(lds_raw + wave * L::kWaveLds);
#pragma unroll
  for (int d = 0; d < D / 16; ++d) *(f32x4 *)(o + n * L::kOStride + 16 * d + 4 * g) = acc[d];
  if (g == 0) {
    ml[wave][0][n] = m;
    ml[wave][1][n] = l;
  }
  __syncthreads();
  constexpr int kVecs = D / 4;  // 4-element vectors of a row
  for (int i = tid; i < t.nr * kVecs; i += kThreads) {
    const int r = i / kVecs, c = (i % kVecs) * 4;
    float mw = ml[0][0][r];
#pragma unroll
    for (int w = 1; w < kWaves; ++w) mw = fmaxf(mw, ml[w][0][r]);
    const float mu = mw == -INFINITY ? 0.0f : mw;
    f32x4 v = {0, 0, 0, 0};
    float sum = 0.0f;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
      const float f = __builtin_amdgcn_exp2f(ml[w][0][r] - mu);
      sum += f * ml[w][1][r];
      v += f * *(const f32x4 *)((const float *)(lds_raw + w * L::kWaveLds) + r * L::kOStride + c);
    }
    const int q = t.r0 + r;
    const int64_t tk = t.t0 + q / a.G, hd = kvh * a.G + q % a.G;
    if (a.splits == 1) {
      const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
      const uint2 w = {pack2<F16>(v[0] * inv, v[1] * inv), pack2<F16>(v[2] * inv, v[3] * inv)};
      *(uint2 *)(a.out.p + tk * a.out.ts + hd * a.out.hs + c) = w;
      if (a.lse && c == 0) a.lse[tk * a.H + hd] = sum == 0.0f ? -INFINITY : (mw + __log2f(sum)) * kLn2;
    } else {
      const int64_t at = (tk * a.H + hd) * a.splits + split;
      *(f32x4 *)(a.part + at * D + c) = v;
      if (c == 0) {
        a.part_ml[2 * at] = mw;
        a.part_ml[2 * at + 1] = sum;
      }
    }
  }
}

// Join the splits' partial results: one wave per (token, head), D / 64 elements a lane.
template <int D, bool F16>
__global__ void __launch_bounds__(kThreads) k_attn_join(AttnArgs a) {
  const int64_t r = (int64_t)blockIdx.x * kWaves + (threadIdx.x >> 6);
  const int lane = threadIdx.x & 63;
  const int64_t tk = r / a.H, hd = r % a.H;
  if (tk >= a.T || tk >= a.b.q_start[a.b.n_seqs]) return;
  const float *ml = a.part_ml + r * a.splits * 2;
  float mw = -INFINITY;
  for (int s = 0; s < a.splits; ++s) mw = fmaxf(mw, ml[2 * s]);
  const float mu = mw == -INFINITY ? 0.0f : mw;
  constexpr int kE = D / 64;
  float v[kE] = {};
  float sum = 0.0f;
  for (int s = 0; s < a.splits; ++s) {
    const float f = __builtin_amdgcn_exp2f(ml[2 * s] - mu);
    sum += f * ml[2 * s + 1];
    const float *p = a.part + (r * a.splits + s) * D + lane * kE;
#pragma unroll
    for (int e = 0; e < kE; ++e) v[e] += f * p[e];
  }
  const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
  uint16_t *o = a.out.p + tk * a.out.ts + hd * a.out.hs + lane * kE;
#pragma unroll
  for (int e = 0; e < kE; ++e) o[e] = (uint16_t)pack2<F16>(v[e] * inv, 0.0f);
  if (a.lse && lane == 0) a.lse[r] = sum == 0.0f ? -INFINITY : (mw + __log2f(sum)) * kLn2;
}

template <int D, bool F16>
hipError_t launch(const AttnArgs &a, hipStream_t s) {
  auto k = k_attn_rows<D, F16>;
  constexpr int lds = Rows<D>::kLds;
  // the attribute belongs to the function on one device: set once for each
  static std::atomic<uint64_t> done{0};
  int dev = 0;
  hipError_t e = hipGetDevice(&dev);
  if (e != hipSuccess) return e;
  if (dev > 63 || !(done.load(std::memory_order_relaxed) >> dev & 1)) {
    e = hipFuncSetAttribute((const void *)k, hipFuncAttributeMaxDynamicSharedMemorySize, lds);
    if (e != hipSuccess) return e;
    if (dev <= 63) done.fetch_or(uint64_t(1) << dev, std::memory_order_relaxed);
  }
  hipLaunchKernelGGL(k, dim3(a.tiles, a.kv.n_kv, a.splits), dim3(kThreads), lds, s, a);
  if (a.splits > 1) {
    auto j = k_attn_join<D, F16>;
    hipLaunchKernelGGL(j, dim3(((int64_t)a.T * a.H + kWaves - 1) / kWaves), dim3(kThreads), 0, s, a);
  }
  return hipGetLastError();
}

}  // namespace

AttnShape attn_shape(int64_t T, int n_seqs, int64_t max_q, int64_t max_kv, int H, int n_kv, int dim) {
  AttnShape s{};
  const int64_t G = H / n_kv;
  s.tiles = (int)(T * G / kAttnRows + n_seqs);
  // tiles that can hold rows, and splits that fill the chip with them
  const int64_t per_seq = (max_q * G + kAttnRows - 1) / kAttnRows;
  const int64_t busy = (per_seq < 1 ? 1 : per_seq) * n_seqs < s.tiles ? (per_seq < 1 ? 1 : per_seq) * n_seqs : s.tiles;
  const int64_t want = 512 / (busy * n_kv < 1 ? 1 : busy * n_kv);
  const int64_t most = (max_kv + kAttnKeys * kWaves - 1) / (kAttnKeys * kWaves);
  int64_t n = want < most ? want : most;
  s.splits = (int)(n < 1 || T * H > 1 << 22 ? 1 : n > 64 ? 64 : n);
  if (s.splits > 1) {
    const size_t rows = (size_t)T * H * s.splits;
    s.off_ml = (rows * dim * 4 + 255) & ~(size_t)255;
    s.ws_bytes = s.off_ml + rows * 8;
  }
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
