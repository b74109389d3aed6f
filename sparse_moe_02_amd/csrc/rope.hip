// Rotary positions of new queries and keys, with the append of keys and values to the
// paged cache, in one launch.
//
// Per pair (a, b) of a head and its frequency f:  theta = pos f,
//     a' = m (a cos theta - b sin theta),   b' = m (a sin theta + b cos theta).
// theta reaches 1e5 rad and more, where binary32 keeps no fraction of a turn: it is formed
// and reduced to a turn in binary64, the sine and cosine of the rest in binary32.
//
// Bound: memory (each element read and written once; 2 bytes each).  A workgroup takes 256
// 16-byte chunks of one token's concatenated heads [q | k | v]: sines and cosines of the
// token's rot_dim / 2 pairs are computed once per workgroup into LDS.  Chunks never straddle
// heads, a head's chunks never straddle workgroups, and all of a workgroup's loads precede
// its stores, so q_out may be q.
#include "paged.hpp"

#pragma clang fp contract(off)

namespace moe {

namespace {

constexpr int kThreads = 256;

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

template <bool F16>
__global__ void __launch_bounds__(kThreads) k_rope_append(RopeArgs a) {
  __shared__ float cs[128], sn[128];
  const int t = blockIdx.x;
  const int tid = threadIdx.x;
  const Batch &b = a.b;
  if (t >= b.q_start[b.n_seqs]) return;  // padding behind the last sequence

  // the token's sequence, position and cache place
  const int seq = wave_find(b.n_seqs, t, [&](int i) { return (int64_t)b.q_start[i]; });
  const int row = batch_row(b, seq);
  const int64_t p = (row < 0 ? 0 : (int64_t)b.kv_len[row]) - b.q_start[seq + 1] + t;
  const double pos = a.pos ? (double)a.pos[t] : (double)p;

  // this thread's chunk of the token's heads
  const int D = a.kv.dim, cph = D / 8;
  const int slot = blockIdx.y * kThreads + tid;
  const int head = slot / cph, i0 = (slot % cph) * 8;
  const int n_kv = a.k.p ? a.kv.n_kv : 0;
  const int kind = head < a.H ? 0 : head < a.H + n_kv ? 1 : head < a.H + 2 * n_kv ? 2 : 3;

  const uint16_t *src = nullptr;
  uint16_t *dst = nullptr;
  if (kind == 0) {
    src = a.q.p + (int64_t)t * a.q.ts + (int64_t)head * a.q.hs;
    dst = a.qo.p + (int64_t)t * a.qo.ts + (int64_t)head * a.qo.hs;
  } else if (kind < 3) {
    const int h = head - a.H - (kind == 2 ? n_kv : 0);
    const Heads &x = kind == 1 ? a.k : a.v;
    src = x.p + (int64_t)t * x.ts + (int64_t)h * x.hs;
    const int64_t col = p >> a.kv.page_shift;
    if (row >= 0 && p >= 0 && col < b.cols) {
      const int page = b.table[(int64_t)row * b.cols + col];
      if ((unsigned)page < (unsigned)a.kv.n_pages)
        dst = (kind == 1 ? a.kv.k : a.kv.v) + (int64_t)page * a.kv.ps +
              (p & ((1 << a.kv.page_shift) - 1)) * a.kv.ts + (int64_t)h * a.kv.hs;
    }
  }
  const int R = a.R, half = R / 2;
  const bool rot = kind < 2 && i0 < R;
  Chunk x, y;
  x.w = y.w = make_uint4(0, 0, 0, 0);
  if (dst) {
    x.w = *(const uint4 *)(src + i0);
    if (rot && !a.interleaved) {
      // element i pairs with i + half (i < half) or i - half
      if (half % 8 == 0) {
        y.w = *(const uint4 *)(src + (i0 < half ? i0 + half : i0 - half));
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int i = i0 + e;
          if (i < R) y.e[e] = src[i < half ? i + half : i - half];
        }
      }
    }
  }
  for (int i = tid; i < half; i += kThreads) {
    const double turns = pos * a.freq[i] * 0.15915494309189533577;  // 1 / (2 pi)
    const float r = (float)(turns - __builtin_rint(turns));
    float s, c;
    sincospif(2.0f * r, &s, &c);
    cs[i] = a.mscale * c;
    sn[i] = a.mscale * s;
  }
  __syncthreads();
  if (!dst) return;
  if (rot) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int i = i0 + e;
      if (i >= R) break;
      if (a.interleaved) {
        if (e & 1) continue;
        const float u = to_f32<F16>(x.e[e]), v = to_f32<F16>(x.e[e + 1]);
        const float c = cs[i / 2], s = sn[i / 2];
        x.e[e] = from_f32<F16>(u * c - v * s);
        x.e[e + 1] = from_f32<F16>(u * s + v * c);
      } else {
        const float u = to_f32<F16>(x.e[e]), v = to_f32<F16>(y.e[e]);
        const bool lo = i < half;
        const float c = cs[lo ? i : i - half], s = sn[lo ? i : i - half];
        x.e[e] = from_f32<F16>(lo ? u * c - v * s : v * s + u * c);
      }
    }
  }
  *(uint4 *)(dst + i0) = x.w;
}

}  // namespace

hipError_t launch_rope_append(const RopeArgs &a, hipStream_t s) {
  const int heads = a.H + (a.k.p ? 2 * a.kv.n_kv : 0);
  if (a.T <= 0 || heads == 0) return hipSuccess;
  const dim3 grid(a.T, (heads * (a.kv.dim / 8) + kThreads - 1) / kThreads);
  if (a.kv.fp16)
    hipLaunchKernelGGL(k_rope_append<true>, grid, dim3(kThreads), 0, s, a);
  else
    hipLaunchKernelGGL(k_rope_append<false>, grid, dim3(kThreads), 0, s, a);
  return hipGetLastError();
}

}  // namespace moe
