// Choice of tokens from logits, with the random numbers given.
//
// Weights w = 2^(y - y_max), y = l log2(e) / temperature in binary64, are held as 64-bit fixed point,
// so that sums are the same in any order.  What is kept is a prefix of the tokens sorted by logit
// (descending) and index, and a token's place in that order is one number (the logit's bits, ordered,
// over the inverted index), so every cut is one such number, and nothing is sorted.
//
//   k_sample_chunks  a workgroup for each 4096 logits: their maximum, and, relative to the power of two
//                    above it, the count and the sum of weights of each eighth of an octave.  Reads
//                    every logit once.  Without filters only the sum.
//   k_sample_cut     a workgroup a row: adds the chunks' bins up, which gives the bin of the first cut
//                    (for top-k, all bins down to it).
//   k_sample_gather  a workgroup a chunk: lists the tokens of that bin, and adds the weights above it.
//   k_sample_pick    a workgroup a row: selects among the listed tokens, 8 bits of their places at a time;
//                    the kept weight of each chunk gives the chunk that u falls into, which is read once
//                    more.  A further cut in another bin is collected here, from the row; where a cut's
//                    bins hold more than kList tokens, each step of the selection reads them from the row.
//
// Short rows and many rows go without the two launches in the middle (`alone`).
//
// Bound: memory and vector units for many rows, latency for few.  256 rows of 131072 fp32: 92 us, of which the chunks
// take 45 (28 without weights, whose 40 instructions a logit are not hidden behind the 134 MB; 39 without the bins'
// atomics); in four launches 96, of which cut 12, gather 23 (the logits again, a quarter of them from the last-level
// cache), pick 21.  One row: 26 to 36 us by what its cut's bins hold, of which 5, 6, 5 to 8 and 10 to 18 are the four
// launches: a chain of loads and barriers in each.  1 and 256 greedy rows 6.6 and 27 (the logits' copy time: 26), without
// filters 11 and 45.  A cut among more than kList tokens costs a read of the row by one workgroup for each step of its
// selection: 1 and 256 flat rows, top-p, 320 and 375, and as long where the cut falls in the last bin (a token of 18
// above 131071 of about 0, top-p 0.999: 330 and 370; min-p, which needs no selection, 95 and 130).
#include "common.hpp"
#include "serve.hpp"

#pragma clang fp contract(off)

namespace moe {

namespace {

constexpr int kChunk = kSampleChunk, kBins = kSampleBins, kPerOctave = 8;
constexpr int kThreads = 256;       // of k_sample_chunks
constexpr int kPick = 1024;         // of k_sample_pick
constexpr int kList = kSampleList;  // tokens that are selected among in LDS
constexpr int kMaxChunks = (1 << 20) / kChunk + 1;
constexpr int kCopies = 4;          // of a chunk's bins, by lane, against conflicts

// 2^(j / 128)
constexpr int kSteps = 128;
__constant__ const double kPow[kSteps] = {
    0x1.0000000000000p+0, 0x1.0163da9fb3335p+0, 0x1.02c9a3e778061p+0, 0x1.04315e86e7f85p+0,
    0x1.059b0d3158574p+0, 0x1.0706b29ddf6dep+0, 0x1.0874518759bc8p+0, 0x1.09e3ecac6f383p+0,
    0x1.0b5586cf9890fp+0, 0x1.0cc922b7247f7p+0, 0x1.0e3ec32d3d1a2p+0, 0x1.0fb66affed31bp+0,
    0x1.11301d0125b51p+0, 0x1.12abdc06c31ccp+0, 0x1.1429aaea92de0p+0, 0x1.15a98c8a58e51p+0,
    0x1.172b83c7d517bp+0, 0x1.18af9388c8deap+0, 0x1.1a35beb6fcb75p+0, 0x1.1bbe084045cd4p+0,
    0x1.1d4873168b9aap+0, 0x1.1ed5022fcd91dp+0, 0x1.2063b88628cd6p+0, 0x1.21f49917ddc96p+0,
    0x1.2387a6e756238p+0, 0x1.251ce4fb2a63fp+0, 0x1.26b4565e27cddp+0, 0x1.284dfe1f56381p+0,
    0x1.29e9df51fdee1p+0, 0x1.2b87fd0dad990p+0, 0x1.2d285a6e4030bp+0, 0x1.2ecafa93e2f56p+0,
    0x1.306fe0a31b715p+0, 0x1.32170fc4cd831p+0, 0x1.33c08b26416ffp+0, 0x1.356c55f929ff1p+0,
    0x1.371a7373aa9cbp+0, 0x1.38cae6d05d866p+0, 0x1.3a7db34e59ff7p+0, 0x1.3c32dc313a8e5p+0,
    0x1.3dea64c123422p+0, 0x1.3fa4504ac801cp+0, 0x1.4160a21f72e2ap+0, 0x1.431f5d950a897p+0,
    0x1.44e086061892dp+0, 0x1.46a41ed1d0057p+0, 0x1.486a2b5c13cd0p+0, 0x1.4a32af0d7d3dep+0,
    0x1.4bfdad5362a27p+0, 0x1.4dcb299fddd0dp+0, 0x1.4f9b2769d2ca7p+0, 0x1.516daa2cf6642p+0,
    0x1.5342b569d4f82p+0, 0x1.551a4ca5d920fp+0, 0x1.56f4736b527dap+0, 0x1.58d12d497c7fdp+0,
    0x1.5ab07dd485429p+0, 0x1.5c9268a5946b7p+0, 0x1.5e76f15ad2148p+0, 0x1.605e1b976dc09p+0,
    0x1.6247eb03a5585p+0, 0x1.6434634ccc320p+0, 0x1.6623882552225p+0, 0x1.68155d44ca973p+0,
    0x1.6a09e667f3bcdp+0, 0x1.6c012750bdabfp+0, 0x1.6dfb23c651a2fp+0, 0x1.6ff7df9519484p+0,
    0x1.71f75e8ec5f74p+0, 0x1.73f9a48a58174p+0, 0x1.75feb564267c9p+0, 0x1.780694fde5d3fp+0,
    0x1.7a11473eb0187p+0, 0x1.7c1ed0130c132p+0, 0x1.7e2f336cf4e62p+0, 0x1.80427543e1a12p+0,
    0x1.82589994cce13p+0, 0x1.8471a4623c7adp+0, 0x1.868d99b4492edp+0, 0x1.88ac7d98a6699p+0,
    0x1.8ace5422aa0dbp+0, 0x1.8cf3216b5448cp+0, 0x1.8f1ae99157736p+0, 0x1.9145b0b91ffc6p+0,
    0x1.93737b0cdc5e5p+0, 0x1.95a44cbc8520fp+0, 0x1.97d829fde4e50p+0, 0x1.9a0f170ca07bap+0,
    0x1.9c49182a3f090p+0, 0x1.9e86319e32323p+0, 0x1.a0c667b5de565p+0, 0x1.a309bec4a2d33p+0,
    0x1.a5503b23e255dp+0, 0x1.a799e1330b358p+0, 0x1.a9e6b5579fdbfp+0, 0x1.ac36bbfd3f37ap+0,
    0x1.ae89f995ad3adp+0, 0x1.b0e07298db666p+0, 0x1.b33a2b84f15fbp+0, 0x1.b59728de5593ap+0,
    0x1.b7f76f2fb5e47p+0, 0x1.ba5b030a1064ap+0, 0x1.bcc1e904bc1d2p+0, 0x1.bf2c25bd71e09p+0,
    0x1.c199bdd85529cp+0, 0x1.c40ab5fffd07ap+0, 0x1.c67f12e57d14bp+0, 0x1.c8f6d9406e7b5p+0,
    0x1.cb720dcef9069p+0, 0x1.cdf0b555dc3fap+0, 0x1.d072d4a07897cp+0, 0x1.d2f87080d89f2p+0,
    0x1.d5818dcfba487p+0, 0x1.d80e316c98398p+0, 0x1.da9e603db3285p+0, 0x1.dd321f301b460p+0,
    0x1.dfc97337b9b5fp+0, 0x1.e264614f5a129p+0, 0x1.e502ee78b3ff6p+0, 0x1.e7a51fbc74c83p+0,
    0x1.ea4afa2a490dap+0, 0x1.ecf482d8e67f1p+0, 0x1.efa1bee615a27p+0, 0x1.f252b376bba97p+0,
    0x1.f50765b6e4540p+0, 0x1.f7bfdad9cbe14p+0, 0x1.fa7c1819e90d8p+0, 0x1.fd3c22b8f71f1p+0};

struct Row {
  double c;          // log2(e) / temperature
  double p, m;       // top_p (1: off), min_p (0: off)
  int k;             // 0: off
  bool greedy, filtered;
};
__device__ __forceinline__ Row read_row(const SampleArgs &a, int r) {
  Row o;
  const float t = a.temperature ? a.temperature[r] : 1.0f;
  o.greedy = !(t > 0.0f);
  o.c = fmax(1.4426950408889634 / (double)t, 1e-300);  // (not 0, so that -infinity stays what it is)
  const int k = a.top_k ? a.top_k[r] : 0;
  o.k = k > 0 && k < a.V ? k : 0;
  const float p = a.top_p ? a.top_p[r] : 1.0f, m = a.min_p ? a.min_p[r] : 0.0f;
  o.p = p < 1.0f ? fmaxf(p, 0.0f) : 1.0;
  o.m = m > 0.0f ? fminf(m, 1.0f) : 0.0;
  o.filtered = o.k > 0 || o.p < 1.0 || o.m > 0.0;
  return o;
}

// 2^(t / 128) times 2^bits, t = 128 (l c - anchor) <= 0, and n = t rounded: 2^x, |x| <= 1/256, by its series
// (off by less than 2^-49), times the table's 2^(j / 128 + bits).  What is below 2^-64 is taken as that (and so is l =
// -infinity), so exponents stay in range and are added as they are; it is 0 as a whole number.
struct Weight {
  double w;
  int n;
  // whole part (the sum with 2^52 rounds; w < 2^52)
  __device__ __forceinline__ uint64_t fixed() const { return (uint64_t)__double_as_longlong(w + 0x1p52) & 0xfffffffffffffull; }
  // number of eighths of an octave below the anchor
  __device__ __forceinline__ int bin() const { return min(kBins - 1, -n >> 4); }
};
static_assert(kSteps / kPerOctave == 16 && kBins <= 64 * kPerOctave, "as Weight::bin has it");
__device__ __forceinline__ Weight weight_at(double t, const double *pow) {
  t = fmax(t, -64.0 * kSteps);
  const double r = t + 0x1.8p52;  // the sum's low bits are t rounded
  const int n = (int)(uint32_t)__double_as_longlong(r);
  const double x = t - (r - 0x1.8p52);
  constexpr double k1 = 0.69314718055994531 / kSteps, k2 = k1 * k1 / 2, k3 = k2 * k1 / 3, k4 = k3 * k1 / 4;
  double s = __builtin_fma(x, k4, k3);
  s = __builtin_fma(x, s, k2);
  s = __builtin_fma(x, s, k1);
  s = __builtin_fma(x, s, 1.0);
  const uint64_t w = (uint64_t)__double_as_longlong(s * pow[n & (kSteps - 1)]);
  return Weight{__longlong_as_double((long long)(w + ((uint64_t)(uint32_t)(n >> 7) << 52))), n};
}
// c: of Row; anchor: in octaves
__device__ __forceinline__ Weight weight_of(float l, double c, double anchor, const double *pow) {
  // (not fused: the anchor is above the rounded product, and far out that is off by whole octaves)
  return weight_at(((double)l * c - anchor) * kSteps, pow);
}
__device__ __forceinline__ void fill_pow(double *pow, int bits) {
  if (threadIdx.x < kSteps) pow[threadIdx.x] = __builtin_amdgcn_ldexp(kPow[threadIdx.x], bits);
}

// Order-preserving bits of a logit (both zeros alike).
__device__ __forceinline__ uint32_t key_of(float l) {
  const uint32_t b = __float_as_uint(l + 0.0f);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}
// A token's place in the descending order: the key over the inverted index, 52 bits.
constexpr int kIndexBits = 20;
constexpr uint32_t kIndexMask = (1u << kIndexBits) - 1;
__device__ __forceinline__ uint64_t place_of(float l, int i) { return (uint64_t)key_of(l) << kIndexBits | (kIndexMask - (uint32_t)i); }
__device__ __forceinline__ int index_of(uint64_t place) { return (int)(kIndexMask - ((uint32_t)place & kIndexMask)); }

__device__ __forceinline__ float logit_of(uint64_t place) {
  const uint32_t key = (uint32_t)(place >> kIndexBits);
  return __uint_as_float(key & 0x80000000u ? key & 0x7fffffffu : ~key);
}

// A row of logits.  Rows may start anywhere; they are read in 16-byte blocks of kVec elements, counted from
// the block that holds the first one (element i is number i + skip), and one by one where a block is
// not the row's alone.
template <int TYPE>
struct Logits {
  static constexpr int kSize = TYPE == 0 ? 4 : 2, kVec = 16 / kSize;
  const uint8_t *base;
  int skip, V;
  __device__ __forceinline__ Logits(const SampleArgs &a, int r) {
    const uint8_t *p = (const uint8_t *)a.logits + (int64_t)r * a.ld * kSize;
    skip = (int)((uintptr_t)p & 15) / kSize;
    base = p - skip * kSize;
    V = a.V;
  }
  // of a block, element e
  __device__ __forceinline__ float raw(u32x4 w, int e) const {
    const uint32_t v = TYPE == 0 ? w[e % 4] : e & 1 ? w[e / 2] >> 16 : w[e / 2] & 0xffffu;
    return TYPE == 0 ? __uint_as_float(v) : TYPE == 1 ? bf16_to_f32((uint16_t)v) : fp16_to_f32((uint16_t)v);
  }
  // numbers n .. n + kVec - 1 (n a multiple of kVec); -infinity outside the row
  __device__ __forceinline__ u32x4 block(int n) const {
    if (n >= skip && n + kVec <= skip + V) return *(const u32x4 *)(base + (int64_t)n * kSize);
    constexpr uint32_t kOut = TYPE == 0 ? 0xff800000u : TYPE == 1 ? 0xff80ff80u : 0xfc00fc00u;
    u32x4 w = {kOut, kOut, kOut, kOut};
#pragma unroll
    for (int e = 0; e < kVec; ++e) {
      if (n + e < skip || n + e >= skip + V) continue;
      if constexpr (TYPE == 0) {
        w[e % 4] = *(const uint32_t *)(base + (int64_t)(n + e) * 4);
      } else {
        const uint32_t v = *(const uint16_t *)(base + (int64_t)(n + e) * 2);
        w[e / 2] = e & 1 ? (w[e / 2] & 0xffffu) | v << 16 : (w[e / 2] & 0xffff0000u) | v;
      }
    }
    return w;
  }
  // as a number; -infinity where it is none
  __device__ __forceinline__ float clean(float l) const { return l == l ? fminf(l, 3.4028234664e38f) : -INFINITY; }
  __device__ __forceinline__ void load(int n, float (&o)[kVec]) const {
    const u32x4 w = block(n);
#pragma unroll
    for (int e = 0; e < kVec; ++e) o[e] = clean(raw(w, e));
  }
};

__device__ __forceinline__ uint64_t shfl_xor_u64(uint64_t v, int d) { return (uint64_t)__shfl_xor((unsigned long long)v, d, 64); }
__device__ __forceinline__ uint64_t wave_sum_u64(uint64_t v) {
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) v += shfl_xor_u64(v, d);
  return v;
}
__device__ __forceinline__ uint64_t wave_max_u64(uint64_t v) {
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) v = max(v, shfl_xor_u64(v, d));
  return v;
}
__device__ __forceinline__ uint64_t wave_scan_u64(uint64_t v) {  // inclusive
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const uint64_t o = (uint64_t)__shfl_up((unsigned long long)v, d, 64);
    if (lane >= d) v += o;
  }
  return v;
}
__device__ __forceinline__ void lds_add(uint64_t *p, uint64_t v) { atomicAdd((unsigned long long *)p, (unsigned long long)v); }

template <int TYPE>
__global__ void __launch_bounds__(kThreads) k_sample_chunks(SampleArgs a) {
  using L = Logits<TYPE>;
  constexpr int kVecs = kChunk / kThreads / L::kVec;  // blocks of a thread
  __shared__ double pow[kSteps];
  __shared__ uint64_t mass[kBins + 1][kCopies];
  __shared__ uint32_t count[kBins + 1][kCopies];
  __shared__ float tops[kThreads / 64];
  __shared__ uint64_t sums[kThreads / 64];
  const int c = blockIdx.x, r = blockIdx.y, tid = threadIdx.x;
  const L logits(a, r);
  float l[kVecs][L::kVec];
  float top = -INFINITY;
#pragma unroll
  for (int q = 0; q < kVecs; ++q) logits.load(c * kChunk + (q * kThreads + tid) * L::kVec, l[q]);
  const Row row = read_row(a, r);
  fill_pow(pow, a.bits);
  if (row.filtered) {
    for (int i = tid; i < kCopies * kBins; i += kThreads) {
      (&mass[0][0])[i] = 0;
      (&count[0][0])[i] = 0;
    }
  }
#pragma unroll
  for (int q = 0; q < kVecs; ++q)
#pragma unroll
    for (int e = 0; e < L::kVec; ++e) top = fmaxf(top, l[q][e]);
  top = wave_max(top);
  if ((tid & 63) == 0) tops[tid >> 6] = top;
  __syncthreads();
  top = fmaxf(fmaxf(tops[0], tops[1]), fmaxf(tops[2], tops[3]));
  SampleChunk *out = a.chunk + (int64_t)r * a.C + c;
  if (row.greedy) {
    uint64_t best = 0;
#pragma unroll
    for (int q = 0; q < kVecs; ++q)
#pragma unroll
      for (int e = 0; e < L::kVec; ++e)
        if (l[q][e] == top && top > -INFINITY)
          best = max(best, place_of(top, c * kChunk + (q * kThreads + tid) * L::kVec + e - logits.skip));
    best = wave_max_u64(best);
    if ((tid & 63) == 0) sums[tid >> 6] = best;
    __syncthreads();
    if (tid == 0) out->best = max(max(sums[0], sums[1]), max(sums[2], sums[3]));
    return;
  }
  const double y0 = (double)top * row.c, anchor = __builtin_ceil(y0);
  uint64_t sum = 0;
  const int copy = tid % kCopies;
  if (top > -INFINITY) {
    // (without a branch a logit, so that several are on their way at once: those that are out go to a bin behind
    // the last)
#pragma unroll
    for (int q = 0; q < kVecs; ++q) {
      uint64_t w[L::kVec];
      int b[L::kVec];
#pragma unroll
      for (int e = 0; e < L::kVec; ++e) {
        const Weight o = weight_of(l[q][e], row.c, anchor, pow);
        w[e] = o.fixed();
        b[e] = l[q][e] == -INFINITY ? kBins : o.bin();
        sum += w[e];
      }
      if (row.filtered) {
#pragma unroll
        for (int e = 0; e < L::kVec; ++e) {
          lds_add(&mass[b[e]][copy], w[e]);
          atomicAdd(&count[b[e]][copy], 1u);
        }
      }
    }
  }
  sum = wave_sum_u64(sum);
  if ((tid & 63) == 0) sums[tid >> 6] = sum;
  __syncthreads();
  if (tid == 0) {
    out->top = y0;
    out->total = sums[0] + sums[1] + sums[2] + sums[3];
  }
  if (!row.filtered) return;
  for (int b = tid; b < kBins; b += kThreads) {
    uint64_t m = 0;
    uint32_t n = 0;
#pragma unroll
    for (int i = 0; i < kCopies; ++i) {
      m += mass[b][i];
      n += count[b][i];
    }
    const int64_t at = ((int64_t)r * a.C + c) * kBins + b;
    a.mass[at] = m;
    a.count[at] = n;
  }
}

// Logits outside these are in none of the row's bins b0 .. b1 (whatever is rounded how).
struct Bounds {
  float least, most;
  __device__ __forceinline__ bool hold(float l) const {
    return l >= least && l <= (most < 3.4028234664e38f ? most : INFINITY) && l > -INFINITY;
  }
};
__device__ __forceinline__ Bounds bounds_of(int b0, int b1, double anchor, double c) {
  // bin b holds 2^t for t from (1/2 - 16 (b + 1)) / 128 up to (1/2 - 16 b) / 128
  constexpr double kStep = 1.0 / kPerOctave, kUp = 0.5 / kSteps;
  auto bound = [&](double y, double way) {
    const double x = (y + way * 1e-3) / c;
    return (float)(x + way * 1e-6 * fabs(x));
  };
  Bounds o;
  o.most = fminf(bound(anchor - b0 * kStep + kUp, 1.0), 3.4028234664e38f);
  o.least = b1 == kBins - 1 ? -INFINITY : bound(anchor - (b1 + 1) * kStep + kUp, -1.0);
  return o;
}

// A chunk's bin among the row's, `shift` octaves above.
__device__ __forceinline__ int row_bin_of(int b, int shift) { return b == kBins - 1 ? b : min(kBins - 1, b + kPerOctave * shift); }
__device__ __forceinline__ int shift_of(double anchor, double chunk) {
  const double d = anchor - chunk;
  return d < 64.0 ? (int)d : 64;
}
// Whether a chunk `shift` octaves below the row, if it has tokens, may have some in the row's bins down to `hi`.  The last
// bin holds what lies anywhere below the others, and such tokens are many: 131071 logits of 0 beside one of 18 have
// 0.2% of the weight.
__device__ __forceinline__ bool reaches_bin(int shift, int hi) { return row_bin_of(0, shift) <= hi; }

// What the threads of k_sample_cut and k_sample_pick share.
struct Shared {
  double pow[kSteps];
  double anchor[kMaxChunks];
  int shift[kMaxChunks];       // octaves of a chunk's anchor below the row's (64: as many or more, weights of 0)
  uint64_t kept[kMaxChunks];   // kept weight of the chunks, then the sums up to each
  int active[kMaxChunks];      // chunks that are read
  uint64_t mass[kBins];        // of the row; then the sums down to each bin
  uint32_t count[kBins];
  uint64_t sel_mass[256];      // of a selection's step
  uint32_t sel_count[256];
  uint64_t red[kPick / 64];
  uint64_t found[3];
  uint64_t left_place[64], left_weight[64];  // the last tokens of a selection
  uint64_t left_before[64], left_above[64];  // what stands above each of them
  int left_n;
  int n, n_active;             // tokens in the list, chunks that are read
};

// The tokens of row bins lo .. hi as a set of (place, weight): in LDS, or read from the row each time.
template <int TYPE>
struct Set {
  using L = Logits<TYPE>;
  const L &logits;
  const Row &row;
  Shared &sh;
  uint64_t *places;
  int lo = 0, hi = -1;  // none
  bool listed = true;
  float least_l, most_l;     // logits outside these are in none of the bins
  uint64_t first, last;      // bounds of the places
  __device__ __forceinline__ Set(const L &logits, const Row &row, Shared &sh, uint64_t *places)
      : logits(logits), row(row), sh(sh), places(places) {}

  // a chunk's bin among the row's
  __device__ __forceinline__ int row_bin(int c, int b) const {
    return row_bin_of(b, sh.shift[c]);
  }
  __device__ __forceinline__ uint64_t scaled(int c, uint64_t m) const { return sh.shift[c] < 64 ? m >> sh.shift[c] : 0; }

  // f(blocks, numbers of their first elements, chunks) for the logits of all active chunks, kAhead blocks a
  // thread at a time, by whole waves: a wave's block is of one chunk (-1: none)
  static constexpr int kPer = kPick * L::kVec / kChunk, kAhead = 4 / kPer;  // chunks of a step, steps in flight
  template <class F>
  __device__ __forceinline__ void scan(F f) const {
    const int tid = threadIdx.x, sub = tid / (kPick / kPer), off = tid % (kPick / kPer) * L::kVec;
    // (the next step's blocks are on their way while f works on this one's)
    u32x4 w[kAhead], next[kAhead];
    int n[kAhead], c[kAhead], cn[kAhead];
    auto ask = [&](int i) {
#pragma unroll
      for (int j = 0; j < kAhead; ++j) {
        const int at = i + j * kPer + sub;
        cn[j] = __builtin_amdgcn_readfirstlane(at < sh.n_active ? sh.active[at] : -1);
        if (cn[j] >= 0) next[j] = logits.block(cn[j] * kChunk + off);
      }
    };
    ask(0);
    for (int i = 0; i < sh.n_active; i += kPer * kAhead) {
#pragma unroll
      for (int j = 0; j < kAhead; ++j) {
        w[j] = next[j];
        c[j] = cn[j];
        n[j] = c[j] * kChunk + off;
      }
      ask(i + kPer * kAhead);
      f(w, n, c);
    }
  }
  // f(logit, number, chunk) for all of them
  template <class F>
  __device__ __forceinline__ void scan_each(F f) const {
    scan([&](const u32x4 (&w)[kAhead], const int (&n)[kAhead], const int (&c)[kAhead]) {
#pragma unroll
      for (int j = 0; j < kAhead; ++j) {
        if (c[j] < 0) continue;
#pragma unroll
        for (int e = 0; e < L::kVec; ++e) f(logits.clean(logits.raw(w[j], e)), n[j] + e, c[j]);
      }
    });
  }
  // whether a logit is in the bins, and its weight
  __device__ __forceinline__ bool in(float l, int c, Weight &w) const {
    if (!(l >= least_l && l <= most_l) || l == -INFINITY) return false;
    w = weight_of(l, row.c, sh.anchor[c], sh.pow);
    const int b = row_bin(c, w.bin());
    return b >= lo && b <= hi;
  }
  template <class F>
  __device__ __forceinline__ void each(F f) const {
    if (listed) {
      constexpr int kAhead = 4;
      for (int i0 = threadIdx.x; i0 < sh.n; i0 += kAhead * kPick) {
        uint64_t place[kAhead];
#pragma unroll
        for (int j = 0; j < kAhead; ++j) place[j] = i0 + j * kPick < sh.n ? places[i0 + j * kPick] : 0;
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
          if (place[j] == 0) continue;
          const int c = (index_of(place[j]) + logits.skip) / kChunk;
          f(place[j], scaled(c, weight_of(logit_of(place[j]), row.c, sh.anchor[c], sh.pow).fixed()), c);
        }
      }
    } else {
      scan_each([&](float l, int n, int c) {
        Weight w;
        if (in(l, c, w)) f(place_of(l, n - logits.skip), scaled(c, w.fixed()), c);
      });
    }
  }
  // bins b0 .. b1, and the chunks that reach them
  __device__ __forceinline__ void range(int b0, int b1, double anchor, int chunks) {
    const int tid = threadIdx.x, lane = tid & 63;
    lo = b0;
    hi = b1;
    const Bounds o = bounds_of(b0, b1, anchor, row.c);
    least_l = o.least;
    most_l = o.most;
    first = (uint64_t)key_of(least_l) << kIndexBits;
    last = (uint64_t)key_of(most_l) << kIndexBits | kIndexMask;
    listed = sh.count[b1] - (b0 > 0 ? sh.count[b0 - 1] : 0) <= (uint32_t)kList;
    __syncthreads();
    if (tid < 64) {  // chunks that reach the bins
      int n = 0;
      for (int c0 = 0; c0 < chunks; c0 += 64) {
        const bool some = c0 + lane < chunks && reaches_bin(sh.shift[c0 + lane], b1) && sh.anchor[c0 + lane] > -INFINITY;
        const uint64_t m = __ballot(some);
        if (some) sh.active[n + __popcll(m & ((uint64_t(1) << lane) - 1))] = c0 + lane;
        n += __popcll(m);
      }
      if (lane == 0) {
        sh.n_active = n;
        sh.n = 0;
      }
    }
    __syncthreads();
  }
  // takes bins b0 .. b1 from the row
  __device__ __forceinline__ void take(int b0, int b1, double anchor, int chunks) {
    const int lane = threadIdx.x & 63;
    range(b0, b1, anchor, chunks);
    if (!listed) return;
    // what lies between the bounds, by a comparison of logits; then those that are in the bins stay: a
    // weight takes 40 instructions, which whole waves would spend on each of their logits
    const Bounds bounds{least_l, most_l};
    scan([&](const u32x4 (&w)[kAhead], const int (&n)[kAhead], const int (&c)[kAhead]) {
      int hits = 0;
#pragma unroll
      for (int j = 0; j < kAhead; ++j) {
        if (c[j] < 0) continue;
#pragma unroll
        for (int e = 0; e < L::kVec; ++e) {
          hits += bounds.hold(logits.raw(w[j], e));
        }
      }
      const int upto = wave_incl_scan(hits), all = __builtin_amdgcn_readlane(upto, 63);
      if (all == 0) return;
      int at = 0;
      if (lane == 0) at = atomicAdd(&sh.n, all);
      at = __builtin_amdgcn_readfirstlane(at) + upto - hits;
      if (hits == 0) return;
#pragma unroll
      for (int j = 0; j < kAhead; ++j) {
        if (c[j] < 0) continue;
#pragma unroll
        for (int e = 0; e < L::kVec; ++e) {
          const float l = logits.raw(w[j], e);
          if (bounds.hold(l)) {
            if (at < kList) places[at] = place_of(logits.clean(l), n[j] + e - logits.skip);
            ++at;
          }
        }
      }
    });
    __syncthreads();
    listed = sh.n <= kList;  // (the bounds may let some more in)
    if (listed) keep_in([&](int i) { return places[i]; });
  }
  // takes bins b0 .. b1, whose tokens and some more are listed
  __device__ __forceinline__ void take_listed(int b0, int b1, double anchor, int chunks, const uint64_t *list, int n) {
    range(b0, b1, anchor, chunks);
    listed = n <= kList;
    if (!listed) return;
    if (threadIdx.x == 0) sh.n = n;
    __syncthreads();
    keep_in([&](int i) { return list[i]; });
  }
  // keeps those of the sh.n tokens that are in the bins
  template <class F>
  __device__ __forceinline__ void keep_in(F from) {
    // (several on their way at once)
    constexpr int kAhead = 8;
    for (int i0 = threadIdx.x; i0 < sh.n; i0 += kAhead * kPick) {
      uint64_t place[kAhead];
#pragma unroll
      for (int j = 0; j < kAhead; ++j) {
        const int i = i0 + j * kPick;
        place[j] = i < sh.n ? from(i) : 0;
      }
#pragma unroll
      for (int j = 0; j < kAhead; ++j) {
        const int i = i0 + j * kPick;
        if (i >= sh.n) break;
        const int c = (index_of(place[j]) + logits.skip) / kChunk;
        Weight w;
        places[i] = in(logit_of(place[j]), c, w) ? place[j] : 0;
      }
    }
    __syncthreads();
  }
};

__device__ __forceinline__ uint64_t block_max(uint64_t v, Shared &sh) {
  const int lane = threadIdx.x & 63;
  v = wave_max_u64(v);
  if (lane == 0) sh.red[threadIdx.x >> 6] = v;
  __syncthreads();
  v = sh.red[lane % (kPick / 64)];
  __syncthreads();
  return wave_max_u64(v);
}

// The least place `at` such that the set's tokens from it on (of those from `least` on) are at least `want` in
// number, or weigh that much, and their weight; all of them where they do not reach that.  8 bits of the places at
// a time, from the first one in which they differ, until at most 64 tokens are left, one a lane.
struct Cut {
  uint64_t at, weight;
};
template <class S>
__device__ __forceinline__ Cut select_from(const S &set, bool by_weight, uint64_t want, uint64_t least, uint32_t tokens, Shared &sh) {
  const int tid = threadIdx.x, lane = tid & 63;
  const uint64_t first = max(set.first, least), differ = first ^ set.last;
  int bits = 64 - __builtin_clzll(differ | 1);  // bits that are not known yet
  uint64_t prefix = set.last >> bits, above = 0;
  while (tokens > 64 && bits > 0) {
    const int rest = max(bits - 8, 0);  // bits below this step's
    for (int i = tid; i < 256; i += kPick) {
      sh.sel_mass[i] = 0;
      sh.sel_count[i] = 0;
    }
    __syncthreads();
    set.each([&](uint64_t place, uint64_t w, int) {
      if (place < least || place >> bits != prefix) return;
      const int b = (int)(place >> rest & ((1u << (bits - rest)) - 1));
      lds_add(&sh.sel_mass[b], w);
      atomicAdd(&sh.sel_count[b], 1u);
    });
    __syncthreads();
    if (tid < 64) {
      // lane i has bins 255 - 4 i down to 252 - 4 i
      uint64_t own[4], sum = 0;
      int low = 256;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int b = 255 - 4 * lane - i;
        own[i] = by_weight ? sh.sel_mass[b] : sh.sel_count[b];
        sum += own[i];
        if (sh.sel_count[b] > 0) low = b;
      }
      const uint64_t upto = wave_scan_u64(sum);
      const uint64_t hit = __ballot(upto >= want), some = __ballot(low < 256);
      uint64_t before = upto - sum;
      int bin = -1;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (bin < 0 && before + own[i] >= want) bin = 255 - 4 * lane - i;
        if (bin < 0) before += own[i];
      }
      // (not reached: the lowest bin that holds anything)
      if (!hit && some) bin = __shfl(low, 63 - __builtin_clzll(some), 64);
      const int cut = hit ? __shfl(bin, __builtin_ctzll(hit), 64) : some ? bin : 0;
      if (hit ? lane == __builtin_ctzll(hit) : lane == 0) {
        sh.found[0] = (uint64_t)cut;
        sh.found[1] = hit ? before : 0;
      }
      uint64_t w = 0;  // weight above the bin
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (255 - 4 * lane - i > cut) w += sh.sel_mass[255 - 4 * lane - i];
      w = wave_sum_u64(w);
      if (lane == 0) {
        sh.found[2] = w;
        if (!hit) sh.found[1] = ~uint64_t(0);
      }
    }
    __syncthreads();
    const uint64_t bin = sh.found[0], before = sh.found[1];
    above += sh.found[2];
    tokens = sh.sel_count[bin];
    __syncthreads();
    prefix = prefix << (bits - rest) | bin;
    bits = rest;
    want = before == ~uint64_t(0) ? before : want - before;  // (not reached: never)
  }
  // the tokens that are left, one a lane
  if (tid == 0) sh.left_n = 0;
  __syncthreads();
  set.each([&](uint64_t place, uint64_t w, int) {
    if (place < least || place >> bits != prefix) return;
    const int at = atomicAdd(&sh.left_n, 1);
    if (at < 64) {
      sh.left_place[at] = place;
      sh.left_weight[at] = w;
    }
  });
  __syncthreads();
  // (each wave compares with its share of them)
  const int n = min(sh.left_n, 64);
  const uint64_t place = lane < n ? sh.left_place[lane] : 0, w = lane < n ? sh.left_weight[lane] : 0;
  if (tid < 64) sh.left_before[tid] = sh.left_above[tid] = 0;
  __syncthreads();
  constexpr int kOwn = 64 / (kPick / 64);
  uint64_t before = 0, weight = 0;
#pragma unroll
  for (int i = 0; i < kOwn; ++i) {
    const int j = (tid >> 6) * kOwn + i;
    if (j >= n) break;
    const uint64_t p = sh.left_place[j], v = sh.left_weight[j];
    if (p > place) {
      before += by_weight ? v : 1;
      weight += v;
    }
  }
  if (weight > 0 || before > 0) {
    lds_add(&sh.left_before[lane], before);
    lds_add(&sh.left_above[lane], weight);
  }
  __syncthreads();
  before = sh.left_before[lane];
  weight = sh.left_above[lane] + above + w;
  const uint64_t own = by_weight ? w : 1;
  uint64_t hit = __ballot(lane < n && before < want && before + own >= want);
  if (!hit) {  // the lowest of them
    uint64_t low = ~wave_max_u64(lane < n ? ~place : 0);
    hit = __ballot(lane < n && place == low);
  }
  __syncthreads();
  if (!hit) return Cut{least, above};
  const int l = __builtin_ctzll(hit);
  return Cut{(uint64_t)__shfl((unsigned long long)place, l, 64), (uint64_t)__shfl((unsigned long long)weight, l, 64)};
}

// The row's largest exponent (-infinity: no tokens); its chunks' anchors and distances.
__device__ __forceinline__ double read_chunks(const SampleArgs &a, int r, Shared &sh) {
  const int tid = threadIdx.x;
  const SampleChunk *chunk = a.chunk + (int64_t)r * a.C;
  auto ordered = [](double y) {  // binary64 numbers as ordered bits
    const uint64_t b = (uint64_t)__double_as_longlong(y + 0.0);
    return b >> 63 ? ~b : b | uint64_t(1) << 63;
  };
  uint64_t most = 0;
  for (int c = tid; c < a.C; c += kPick) {
    const double y = chunk[c].top;
    sh.anchor[c] = __builtin_ceil(y);
    most = max(most, ordered(y));
  }
  most = block_max(most, sh);
  const double y0 = __longlong_as_double((long long)(most >> 63 ? most & ~(uint64_t(1) << 63) : ~most));
  const double anchor = __builtin_ceil(y0);
  for (int c = tid; c < a.C; c += kPick) sh.shift[c] = shift_of(anchor, sh.anchor[c]);
  __syncthreads();
  return y0;
}
// The chunks' bins, N a thread at a time from number i0 on.
template <int N>
struct Bins {
  static constexpr int kAhead = N;
  uint32_t n[kAhead];
  uint64_t m[kAhead];
  __device__ __forceinline__ void load(const SampleArgs &a, int r, int i0) {
    const uint64_t *mass = a.mass + (int64_t)r * a.C * kBins;
    const uint32_t *count = a.count + (int64_t)r * a.C * kBins;
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      const int i = i0 + j * kPick;
      n[j] = 0;
      if (i < a.C * kBins) {
        n[j] = count[i];
        m[j] = mass[i];
      }
    }
  }
};
// f(chunk, bin of the chunk, count, weights), of those that hold tokens; b: the first ones
template <int N, class F>
__device__ __forceinline__ void each_bin(const SampleArgs &a, int r, Bins<N> &b, F f) {
  for (int i0 = threadIdx.x; i0 < a.C * kBins; i0 += N * kPick) {
    if (i0 >= N * kPick) b.load(a, r, i0);
#pragma unroll
    for (int j = 0; j < N; ++j)
      if (b.n[j] > 0) f((i0 + j * kPick) / kBins, (i0 + j * kPick) % kBins, b.n[j], b.m[j]);
  }
}
// the first bin down to which `enough` holds
template <class F>
__device__ __forceinline__ int first_bin(F enough) {
  const int lane = threadIdx.x & 63;
  for (int b = 0; b < kBins; b += 64) {
    const uint64_t yes = __ballot(enough(b + lane));
    if (yes) return b + (int)__builtin_ctzll(yes);
  }
  return kBins - 1;
}
static_assert(kBins % 64 == 0, "bins are read by whole waves");
// A share of a total as a whole number, at least 1.
__device__ __forceinline__ uint64_t share_of(double p, uint64_t total) {
  return max(min((uint64_t)__builtin_ceil(p * (double)total), total), uint64_t(1));
}
// The bins of the top-k cut: from the first one on where they hold few tokens, so that a top-p cut among them
// needs no others.
__device__ __forceinline__ void top_k_bins(const Shared &sh, int k, int &lo, int &hi) {
  hi = first_bin([&](int b) { return sh.count[b] >= (uint32_t)k; });
  lo = sh.count[hi] <= (uint32_t)kList ? 0 : hi;
}
__device__ __forceinline__ double floor_of(const Row &row, double y0) { return row.m > 0.0 ? y0 + log2(row.m) : -INFINITY; }

// Adds the chunks' bins up (into sh.mass and sh.count, which are 0 before) down to each; the bins of the first
// cut (hi < lo: none).
template <int N>
__device__ __forceinline__ void cut_bins(const SampleArgs &a, int r, const Row &row, Shared &sh, Bins<N> &bins, double y0, int &lo, int &hi) {
  const int tid = threadIdx.x, lane = tid & 63;
  each_bin(a, r, bins, [&](int c, int b, uint32_t n, uint64_t m) {
    const int s = sh.shift[c];
    b = row_bin_of(b, s);
    atomicAdd(&sh.count[b], n);
    lds_add(&sh.mass[b], s < 64 ? m >> s : 0);
  });
  __syncthreads();
  if (tid < 64) {  // sums down to each bin
    constexpr int kOwn = kBins / 64;
    uint64_t m[kOwn], n[kOwn], ms = 0, ns = 0;
#pragma unroll
    for (int i = 0; i < kOwn; ++i) {
      m[i] = ms += sh.mass[lane * kOwn + i];
      n[i] = ns += sh.count[lane * kOwn + i];
    }
    const uint64_t mb = wave_scan_u64(ms) - ms, nb = wave_scan_u64(ns) - ns;
#pragma unroll
    for (int i = 0; i < kOwn; ++i) {
      sh.mass[lane * kOwn + i] = mb + m[i];
      sh.count[lane * kOwn + i] = (uint32_t)(nb + n[i]);
    }
  }
  __syncthreads();
  lo = 0;
  hi = -1;
  const uint64_t total = sh.mass[kBins - 1];
  if (row.k > 0 && (uint32_t)row.k < sh.count[kBins - 1]) {
    top_k_bins(sh, row.k, lo, hi);
  } else if (row.p < 1.0) {
    lo = hi = first_bin([&](int i) { return sh.mass[i] >= share_of(row.p, total); });
  } else if (row.m > 0.0) {
    lo = hi = weight_at((floor_of(row, y0) - __builtin_ceil(y0)) * kSteps, sh.pow).bin();
  }
}

__global__ void __launch_bounds__(kPick) k_sample_cut(SampleArgs a) {
  __shared__ Shared sh;
  const int r = blockIdx.x, tid = threadIdx.x;
  const Row row = read_row(a, r);
  if (row.greedy || !row.filtered) return;
  Bins<7> bins;  // (asked for before the chunks' maxima are waited for)
  bins.load(a, r, tid);
  fill_pow(sh.pow, a.bits);
  for (int i = tid; i < kBins; i += kPick) {
    sh.mass[i] = 0;
    sh.count[i] = 0;
  }
  const double y0 = read_chunks(a, r, sh);
  SampleRow *out = a.row + r;
  if (y0 == -INFINITY) {
    if (tid == 0) {
      out->lo = 0;
      out->hi = -1;
    }
    return;
  }
  int lo, hi;
  cut_bins(a, r, row, sh, bins, y0, lo, hi);
  if (tid < kBins) {
    out->mass[tid] = sh.mass[tid];
    out->count[tid] = sh.count[tid];
  }
  if (tid == 0) {
    out->lo = lo;
    out->hi = hi;
    out->n = 0;
  }
}

template <int TYPE>
__global__ void __launch_bounds__(kThreads) k_sample_gather(SampleArgs a) {
  using L = Logits<TYPE>;
  constexpr int kVecs = kChunk / kThreads / L::kVec;
  __shared__ uint64_t sums[kThreads / 64];
  __shared__ double tops[kThreads / 64];
  __shared__ int hits[kThreads / 64], base;
  const int c = blockIdx.x, r = blockIdx.y, tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const Row row = read_row(a, r);
  if (row.greedy || !row.filtered) return;
  SampleRow *out = a.row + r;
  const int lo = out->lo, hi = out->hi;
  const L logits(a, r);
  u32x4 w[kVecs];
#pragma unroll
  for (int q = 0; q < kVecs; ++q) w[q] = logits.block(c * kChunk + (q * kThreads + tid) * L::kVec);
  const SampleChunk *chunk = a.chunk + (int64_t)r * a.C;
  double y0 = -INFINITY;
  for (int i = tid; i < a.C; i += kThreads) y0 = fmax(y0, chunk[i].top);
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) y0 = fmax(y0, __shfl_xor(y0, d, 64));
  const double mine = chunk[c].top;
  const int64_t at = ((int64_t)r * a.C + c) * kBins;
  const uint32_t n = tid < kBins ? a.count[at + tid] : 0;
  const uint64_t m = tid < kBins ? a.mass[at + tid] : 0;
  if (lane == 0) tops[wave] = y0;
  if (hi < lo) return;
  __syncthreads();
  y0 = fmax(fmax(tops[0], tops[1]), fmax(tops[2], tops[3]));
  const double anchor = __builtin_ceil(y0);
  const int shift = mine == -INFINITY ? 64 : shift_of(anchor, __builtin_ceil(mine));
  const uint64_t sum = wave_sum_u64(n > 0 && shift < 64 && row_bin_of(tid, shift) < lo ? m >> shift : 0);
  const Bounds bounds = bounds_of(lo, hi, anchor, row.c);
  const bool reaches = mine > -INFINITY && reaches_bin(shift, hi);
  int some = 0;
  if (reaches) {
#pragma unroll
    for (int q = 0; q < kVecs; ++q)
#pragma unroll
      for (int e = 0; e < L::kVec; ++e) some += bounds.hold(logits.raw(w[q], e));
  }
  const int upto = wave_incl_scan(some);
  if (lane == 63) hits[wave] = upto;
  if (lane == 0) sums[wave] = sum;
  __syncthreads();
  const int all = hits[0] + hits[1] + hits[2] + hits[3];
  if (tid == 0) {
    a.kept[(int64_t)r * a.C + c] = sums[0] + sums[1] + sums[2] + sums[3];
    if (all > 0) base = atomicAdd(&out->n, all);
  }
  if (all == 0) return;
  __syncthreads();
  int to = base + upto - some;
  for (int i = 0; i < wave; ++i) to += hits[i];
  if (some == 0) return;
  uint64_t *list = a.list + (int64_t)r * a.room;
#pragma unroll
  for (int q = 0; q < kVecs; ++q)
#pragma unroll
    for (int e = 0; e < L::kVec; ++e) {
      const float l = logits.raw(w[q], e);
      if (bounds.hold(l)) {
        if (to < a.room) list[to] = place_of(logits.clean(l), c * kChunk + (q * kThreads + tid) * L::kVec + e - logits.skip);
        ++to;
      }
    }
}

// ALONE: without k_sample_cut and k_sample_gather before it, whose work it does itself.
template <int TYPE, bool ALONE>
__global__ void __launch_bounds__(kPick) k_sample_pick(SampleArgs a) {
  using L = Logits<TYPE>;
  extern __shared__ __align__(16) uint8_t lds_raw[];
  __shared__ Shared sh;
  const int r = blockIdx.x, tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const Row row = read_row(a, r);
  const L logits(a, r);
  const SampleChunk *chunk = a.chunk + (int64_t)r * a.C;
  fill_pow(sh.pow, a.bits);
  // asked for here, so that these are not waited for one after the other
  const float u0 = a.u[r];
  const SampleRow *in = a.row + r;
  int lo = 0, hi = -1, listed = 0;
  uint64_t mass = 0, kept = 0;
  uint32_t count = 0;
  Bins<4> bins;
  if (row.filtered && !row.greedy && ALONE) {
    bins.load(a, r, tid);
    if (tid < kBins) {
      sh.mass[tid] = 0;
      sh.count[tid] = 0;
    }
  } else if (row.filtered && !row.greedy) {
    lo = in->lo;
    hi = in->hi;
    listed = in->n;
    if (tid < kBins) {
      mass = in->mass[tid];
      count = in->count[tid];
    }
    if (tid < a.C) kept = a.kept[(int64_t)r * a.C + tid];
  }
  static_assert(kBins <= kPick && kMaxChunks <= kPick, "one a thread");

  if (row.greedy) {
    uint64_t best = 0;
    for (int c = tid; c < a.C; c += kPick) best = max(best, chunk[c].best);
    best = block_max(best, sh);
    if (tid == 0) {
      a.token[r] = best ? index_of(best) : -1;
      if (a.prob) a.prob[r] = best ? 1.0f : 0.0f;
    }
    return;
  }
  const double y0 = read_chunks(a, r, sh), anchor = __builtin_ceil(y0);
  if (y0 == -INFINITY) {
    if (tid == 0) {
      a.token[r] = -1;
      if (a.prob) a.prob[r] = 0.0f;
    }
    return;
  }

  uint64_t least = 0;          // places that are kept are at least this
  const double least_y = floor_of(row, y0);
  double floor = -INFINITY;    // and exponents this
  auto above_floor = [&](float l) { return (double)l * row.c >= floor; };
  if (!row.filtered) {
    for (int c = tid; c < a.C; c += kPick) sh.kept[c] = sh.shift[c] < 64 ? chunk[c].total >> sh.shift[c] : 0;
  } else {
    if constexpr (ALONE) {
      cut_bins(a, r, row, sh, bins, y0, lo, hi);
    } else if (tid < kBins) {
      sh.mass[tid] = mass;
      sh.count[tid] = count;
    }
    Set<TYPE> set(logits, row, sh, (uint64_t *)lds_raw);
    __syncthreads();
    if (hi >= lo && ALONE) set.take(lo, hi, anchor, a.C);
    else if (hi >= lo) set.take_listed(lo, hi, anchor, a.C, a.list + (int64_t)r * a.room, listed);
    auto mass_above = [&](int b) { return b > 0 ? sh.mass[b - 1] : 0; };
    auto count_above = [&](int b) { return b > 0 ? sh.count[b - 1] : 0u; };
    auto held = [&] { return sh.count[set.hi] - count_above(set.lo); };  // tokens of the set
    auto has = [&](int b) { return set.lo <= b && b <= set.hi; };

    int cut = kBins;  // the bin of the cut
    uint64_t total = sh.mass[kBins - 1];
    if (row.k > 0 && (uint32_t)row.k < sh.count[kBins - 1]) {  // (k_sample_cut has taken its bins)
      cut = set.hi;
      const Cut o = select_from(set, false, (uint64_t)row.k - count_above(set.lo), 0, held(), sh);
      least = o.at;
      total = mass_above(set.lo) + o.weight;
    }
    if (row.p < 1.0) {
      const uint64_t want = share_of(row.p, total);
      const int b = min(cut, first_bin([&](int i) { return sh.mass[i] >= want; }));
      if (!has(b)) set.take(b, b, anchor, a.C);
      const uint64_t over = mass_above(set.lo);
      least = max(least, select_from(set, true, want > over ? want - over : 1, least, held(), sh).at);
      cut = b;
    }
    if (row.m > 0.0) {
      floor = least_y;
      const int b = weight_at((floor - anchor) * kSteps, sh.pow).bin();
      if (b <= cut && !has(b)) set.take(b, b, anchor, a.C);
    }
    const bool none = set.hi < 0;  // no cut: all bins
    if (!none && set.lo == lo && !ALONE) {
      if (tid < a.C) sh.kept[tid] = kept;
      __syncthreads();
    } else {
      for (int c = tid; c < a.C; c += kPick) sh.kept[c] = 0;
      __syncthreads();
      bins.load(a, r, tid);
      each_bin(a, r, bins, [&](int c, int b, uint32_t, uint64_t m) {
        if (none || set.row_bin(c, b) < set.lo) lds_add(&sh.kept[c], set.scaled(c, m));
      });
    }
    if (!none && set.listed) {
      set.each([&](uint64_t place, uint64_t w, int c) {
        if (place >= least && above_floor(logit_of(place))) lds_add(&sh.kept[c], w);
      });
    } else if (!none) {  // (a wave's logits are of one chunk)
      uint64_t sum = 0;
      int at = -1;
      auto flush = [&] {
        const uint64_t v = wave_sum_u64(sum);
        if (lane == 0 && v > 0) lds_add(&sh.kept[at], v);
        sum = 0;
      };
      set.scan_each([&](float l, int n, int c) {
        if (c != at) {
          if (at >= 0) flush();
          at = c;
        }
        Weight w;
        if (set.in(l, c, w) && place_of(l, n - logits.skip) >= least && above_floor(l)) sum += set.scaled(c, w.fixed());
      });
      if (at >= 0) flush();
    }
  }
  __syncthreads();

  // sums up to each chunk
  if (wave == 0) {
    uint64_t before = 0;
    for (int c0 = 0; c0 < a.C; c0 += 64) {
      const uint64_t v = c0 + lane < a.C ? sh.kept[c0 + lane] : 0;
      const uint64_t upto = before + wave_scan_u64(v);
      if (c0 + lane < a.C) sh.kept[c0 + lane] = upto;
      before = (uint64_t)__shfl((unsigned long long)upto, 63, 64);
    }
  }
  __syncthreads();
  const uint64_t total = sh.kept[a.C - 1];
  const double u = u0 > 0.0f ? fminf(u0, 1.0f) : 0.0;
  const uint64_t want = min((uint64_t)(u * (double)total), total - 1);  // (the first sum above it is wanted)
  int c = 0;
  for (int c0 = 0; c0 < a.C; c0 += 64) {
    const uint64_t m = __ballot(c0 + lane < a.C && sh.kept[min(c0 + lane, a.C - 1)] > want);
    if (m) {
      c = c0 + (int)__builtin_ctzll(m);
      break;
    }
  }
  // in the chunk, in its own weights
  const int shift = sh.shift[c];
  const double from = sh.anchor[c];
  uint64_t target = (want - (c > 0 ? sh.kept[c - 1] : 0)) << shift;
  constexpr int kHave = kChunk / L::kVec;  // threads with logits
  float l[L::kVec];
  uint64_t w[L::kVec], mine = 0, upto = 0, before = 0, all = 0;
  const int n = c * kChunk + tid * L::kVec;
#pragma unroll
  for (int e = 0; e < L::kVec; ++e) l[e] = -INFINITY;
  if (tid < kHave) logits.load(n, l);
  for (int pass = 0; pass < 2 && all == 0; ++pass) {
    mine = 0;
#pragma unroll
    for (int e = 0; e < L::kVec; ++e) {
      const bool keep = l[e] > -INFINITY && place_of(l[e], n + e - logits.skip) >= least && above_floor(l[e]);
      w[e] = keep ? weight_of(l[e], row.c, from, sh.pow).fixed() : 0;
      mine += w[e];
    }
    upto = wave_scan_u64(mine);
    __syncthreads();
    if (lane == 63) sh.red[wave] = upto;
    __syncthreads();
    before = all = 0;
    for (int i = 0; i < kPick / 64; ++i) {
      if (i < wave) before += sh.red[i];
      all += sh.red[i];
    }
    // (the chunk has kept weight; a token that lies within a rounding of its bin's edge could be in the bins
    // that are kept and yet behind the cut, and alone: then the chunk's tokens are taken as they are)
    least = 0;
    floor = -INFINITY;
  }
  if (all == 0) return;
  target = min(target, all - 1);
  before += upto - mine;
  if (target >= before && target < before + mine) {
    uint64_t sum = before;
#pragma unroll
    for (int e = 0; e < L::kVec; ++e) {
      if (target >= sum && target < sum + w[e]) {
        a.token[r] = n + e - logits.skip;
        if (a.prob) a.prob[r] = (float)(__builtin_amdgcn_ldexp(weight_of(l[e], row.c, from, sh.pow).w, -shift) / (double)total);
      }
      sum += w[e];
    }
  }
}

template <int TYPE, bool ALONE>
hipError_t pick(const SampleArgs &a, hipStream_t s) {
  static std::atomic<uint64_t> done{0};
  constexpr int lds = kList * 8;
  const hipError_t e = allow_lds(k_sample_pick<TYPE, ALONE>, lds, done);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL((k_sample_pick<TYPE, ALONE>), dim3(a.R), dim3(kPick), lds, s, a);
  return hipGetLastError();
}

// Whether k_sample_pick goes alone behind the first launch: for short rows, whose two launches in between take longer
// than reading them once more with one workgroup, and for many, which fill the chip by themselves.  us alone and not, rows
// with top-p: 1 of 1000 17.8 and 23.2, 1 of 32000 21.4 and 24.2, but 1 of 131072 31.5 and 26.3; 48 of 64000 40 and 37, of
// 131072 64 and 53; 96 of 64000 46.1 and 46.8, of 131072 74 and 69; 192 of 64000 60 and 68, of 131072 92 and 100; 256 of
// 131072 101 and 112.
bool alone(const SampleArgs &a) { return a.C <= 8 || 5 * a.C <= a.R; }

template <int TYPE>
hipError_t launch(const SampleArgs &a, hipStream_t s) {
  hipLaunchKernelGGL((k_sample_chunks<TYPE>), dim3(a.C, a.R), dim3(kThreads), 0, s, a);
  const bool filters = a.top_k || a.top_p || a.min_p;  // (otherwise no row has any)
  if (!filters || alone(a)) return pick<TYPE, true>(a, s);
  hipLaunchKernelGGL(k_sample_cut, dim3(a.R), dim3(kPick), 0, s, a);
  hipLaunchKernelGGL((k_sample_gather<TYPE>), dim3(a.C, a.R), dim3(kThreads), 0, s, a);
  return pick<TYPE, false>(a, s);
}

}  // namespace

hipError_t launch_sample(const SampleArgs &a, hipStream_t s) {
  if (a.R <= 0) return hipSuccess;
  switch (a.type) {
    case 0: return launch<0>(a, s);
    case 1: return launch<1>(a, s);
    case 2: return launch<2>(a, s);
  }
  return hipErrorInvalidValue;
}

}  // namespace moe
