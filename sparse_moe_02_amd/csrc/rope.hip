// Rotary positions of new queries and keys, with the append of keys and values to the
// paged cache, in one launch.
//
// Per pair (a, b) of a head and its frequency f:  theta = pos f,
//     a' = m (a cos theta - b sin theta),   b' = m (a sin theta + b cos theta).
// theta reaches 1e5 rad and more, where binary32 keeps no fraction of a turn: it is formed
// and reduced to a turn in binary64, the sine and cosine of the rest in binary32.
//
// Bound: memory (each element read and written once; 2 bytes each).  A workgroup takes 16-byte
// chunks of one token's concatenated heads [q | k | v]: sines and cosines of the token's
// rot_dim / 2 pairs are computed once per workgroup into LDS.  Chunks never straddle heads, a
// head's chunks never straddle workgroups, and all of a workgroup's loads precede its stores, so
// q_out may be q.  The data loads do not wait for the token's sequence, and a large call's threads
// take three chunks each: 4096 tokens of 16 + 2 + 2 heads of 256 take 17.0 us, 4.9 TB/s (one
// chunk a thread 23.1, two 22.0, four 18.0).  16 tokens: 4.3 us, the launch and four dependent loads.
#include "paged.hpp"

#pragma clang fp contract(off)

namespace moe {

namespace {

constexpr int kThreads = 256;
constexpr int kMany = 3;    // chunks a thread of a large call
constexpr int kFew = 1024;  // workgroups of one chunk a thread that leave room on the chip

template <bool F16>
__device__ __forceinline__ float to_f32(uint16_t v) {
  return F16 ? fp16_to_f32(v) : bf16_to_f32(v);
}
template <bool F16>
__device__ __forceinline__ uint16_t from_f32(float v) {
  return F16 ? __builtin_bit_cast(uint16_t, (_Float16)v) : f32_to_bf16(v);
}

union Chunk {
  uint4 w;
  uint16_t e[8];
};

// How the elements of a pair lie: half a rotation apart in whole chunks, side by side, or half
// a rotation apart anyhow.
enum class Pairs { Chunks, Adjacent, Any };

// kPer chunks a thread.
template <bool F16, int kPer, Pairs kPairs>
__global__ void __launch_bounds__(kThreads) k_rope_append(RopeArgs a) {
  __shared__ float cs[128], sn[128];
  const int t = blockIdx.x;
  const int tid = threadIdx.x;
  const Batch &b = a.b;
  const int shift = a.kv.dim == 256 ? 5 : a.kv.dim == 128 ? 4 : 3;  // log2 of a head's chunks
  const int R = a.R, half = R / 2;
  const int n_kv = a.k.p ? a.kv.n_kv : 0;
  const int heads = a.H + 2 * n_kv;

  // this thread's chunks of the token's heads, read before anything is known of its sequence,
  // and without branches, which would wait for the loads one by one
  uint4 x[kPer], y[kPer];
  int head[kPer], kind[kPer];  // kind: q, k, v
  const int i0 = tid % (1 << shift) * 8;
  const bool in_rot = i0 < R;
#pragma unroll
  for (int j = 0; j < kPer; ++j) {
    const int h0 = min(((int)(blockIdx.y * kPer + j) * kThreads + tid) >> shift, heads - 1);
    kind[j] = h0 < a.H ? 0 : h0 < a.H + n_kv ? 1 : 2;
    head[j] = h0 - (kind[j] > 0 ? a.H : 0) - (kind[j] > 1 ? n_kv : 0);
    const Heads h = kind[j] == 0 ? a.q : kind[j] == 1 ? a.k : a.v;
    const uint16_t *src = h.p + (int64_t)t * h.ts + (int64_t)head[j] * h.hs;
    x[j] = *(const uint4 *)(src + i0);
    // element i pairs with i + half (i < half) or i - half
    if (kPairs == Pairs::Chunks) y[j] = *(const uint4 *)(src + (!in_rot ? i0 : i0 < half ? i0 + half : i0 - half));
    if (kPairs == Pairs::Any) {
      Chunk c;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int i = i0 + e;
        c.e[e] = src[i >= R ? i : i < half ? i + half : i - half];
      }
      y[j] = c.w;
    }
  }
  // the token's sequence, position and cache place
  int row, len, end;  // table row, its length, first token behind the sequence
  if (b.n_seqs > 1 && b.n_seqs <= 64) {
    // every sequence in a lane: one step less in the chain of loads (2777 tokens of 48 sequences 14.9
    // us, 15.2 the other way; one sequence's numbers come faster as scalars, 17.6 and 19.7)
    const int lane = tid & 63, i = min(lane, b.n_seqs - 1);
    const int from = b.q_start[i], to = b.q_start[i + 1], r = batch_row(b, i), n = b.kv_len[max(r, 0)];
    const int seq = max(0, 63 - (int)__builtin_clzll(__ballot(lane < b.n_seqs && from <= t) | 1));
    if (t >= __builtin_amdgcn_readlane(to, b.n_seqs - 1)) return;  // padding behind the last sequence
    row = __builtin_amdgcn_readlane(r, seq);
    len = __builtin_amdgcn_readlane(n, seq);
    end = __builtin_amdgcn_readlane(to, seq);
  } else {
    if (t >= b.q_start[b.n_seqs]) return;
    const int seq = wave_find(b.n_seqs, t, [&](int i) { return (int64_t)b.q_start[i]; });
    row = batch_row(b, seq);
    len = b.kv_len[max(row, 0)];
    end = b.q_start[seq + 1];
  }
  const int64_t p = (row < 0 ? 0 : (int64_t)len) - end + t;
  const int64_t col = p >> a.kv.page_shift;
  int page = -1;
  if (n_kv && row >= 0 && p >= 0 && col < b.cols) page = b.table[(int64_t)row * b.cols + col];
  const double pos = a.pos ? (double)a.pos[t] : (double)p;
  for (int i = tid; i < half; i += kThreads) {
    const double turns = pos * a.freq[i] * 0.15915494309189533577;  // 1 / (2 pi)
    const float r = (float)(turns - __builtin_rint(turns));
    float s, c;
    sincospif(2.0f * r, &s, &c);
    cs[i] = a.mscale * c;
    sn[i] = a.mscale * s;
  }
  __syncthreads();
  const bool stored = (unsigned)page < (unsigned)a.kv.n_pages;
  const int64_t place = stored ? page * a.kv.ps + (p & ((1 << a.kv.page_shift) - 1)) * a.kv.ts : 0;
  // a chunk's pairs are the same in every head
  float c8[8], s8[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const int i = i0 + e, pair = kPairs == Pairs::Adjacent ? i / 2 : i < half ? i : i - half;
    c8[e] = i < R ? cs[pair] : 1.0f;
    s8[e] = i < R ? (i < half || kPairs == Pairs::Adjacent ? sn[pair] : -sn[pair]) : 0.0f;
  }
#pragma unroll
  for (int j = 0; j < kPer; ++j) {
    if (((int)(blockIdx.y * kPer + j) * kThreads + tid) >> shift >= heads || (kind[j] > 0 && !stored)) continue;
    Chunk u, v;
    u.w = x[j];
    if (kind[j] < 2 && in_rot) {
      if (kPairs == Pairs::Adjacent) {
#pragma unroll
        for (int e = 0; e < 8; e += 2) {
          const float p0 = to_f32<F16>(u.e[e]), p1 = to_f32<F16>(u.e[e + 1]);
          const uint16_t q0 = from_f32<F16>(p0 * c8[e] - p1 * s8[e]), q1 = from_f32<F16>(p0 * s8[e] + p1 * c8[e]);
          u.e[e] = i0 + e < R ? q0 : u.e[e];
          u.e[e + 1] = i0 + e < R ? q1 : u.e[e + 1];
        }
      } else {
        v.w = y[j];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const uint16_t q = from_f32<F16>(to_f32<F16>(u.e[e]) * c8[e] - to_f32<F16>(v.e[e]) * s8[e]);
          u.e[e] = i0 + e < R ? q : u.e[e];
        }
      }
    }
    uint16_t *dst = kind[j] == 0 ? a.qo.p + (int64_t)t * a.qo.ts + (int64_t)head[j] * a.qo.hs
                                 : (kind[j] == 1 ? a.kv.k : a.kv.v) + place + (int64_t)head[j] * a.kv.hs;
    *(uint4 *)(dst + i0) = u.w;
  }
}

template <bool F16, Pairs kPairs>
void launch(const RopeArgs &a, int per, int parts, hipStream_t s) {
  const dim3 grid(a.T, parts);
  if (per == 1)
    hipLaunchKernelGGL((k_rope_append<F16, 1, kPairs>), grid, dim3(kThreads), 0, s, a);
  else
    hipLaunchKernelGGL((k_rope_append<F16, kMany, kPairs>), grid, dim3(kThreads), 0, s, a);
}
template <bool F16>
void launch(const RopeArgs &a, int per, int parts, hipStream_t s) {
  if (a.interleaved)
    launch<F16, Pairs::Adjacent>(a, per, parts, s);
  else if (a.R % 16 == 0)
    launch<F16, Pairs::Chunks>(a, per, parts, s);
  else
    launch<F16, Pairs::Any>(a, per, parts, s);
}

}  // namespace

hipError_t launch_rope_append(const RopeArgs &a, hipStream_t s) {
  const int heads = a.H + (a.k.p ? 2 * a.kv.n_kv : 0);
  if (a.T <= 0 || heads == 0) return hipSuccess;
  const int chunks = heads * (a.kv.dim / 8), blocks = (chunks + kThreads - 1) / kThreads;
  const int per = (int64_t)a.T * blocks <= kFew ? 1 : kMany;
  if (a.kv.fp16)
    launch<true>(a, per, (blocks + per - 1) / per, s);
  else
    launch<false>(a, per, (blocks + per - 1) / per, s);
  return hipGetLastError();
}

}  // namespace moe
