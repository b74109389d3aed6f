// Products of few rows with 4-bit weights ("Optimizing on-device inference for Apple Silicon",
// section "Decode > Optimize the one-row weight path").
//
//     out[t][n] = sum_g s[n][g] (sum_{k in g} code x) + b[n][g] (sum_{k in g} x),  groups of 64.
//
// Bound: memory, 0.5625 bytes a weight, read once.  Even a single row goes over the matrix units: 8 codes are turned
// into an operand's registers with 8 vector instructions for up to 16 rows of x at once, where dot products
// need 4 more for each row.  Codes enter as 16 + code, which is exact in either type (the mantissa's top bits), so a
// group's products start from a sum of zero and are scaled in binary32:
//     acc += s r + (b - 16 s) X,   r = sum x (16 + code),  X = sum x,
// where a larger offset (128 + code) would cost eight times the rounding.  int8 rows take the codes
// as bytes, and r and X are exact.
//
// Rows of x are the products' rows and weight rows their columns, so that a lane's results belong to one weight row
// and need one scale and one bias a group: those of four groups come with one 2-byte load a lane each.  (With
// weight rows as the products' rows a lane needs four of them, in 8-byte loads that 16 lanes share: these alone
// took 30 of 64 us for 8 rows of 2048 -> 131072.)
//
// Measured: 8 rows of 2048 -> 131072, fp32 out, 34 to 37.5 us, 155 MB at 4.1 to 4.6 TB/s, vector units busy for three
// quarters of the cycles (they turn codes into operands); one row of 2048 -> 5120 5.5 (launch, a chain of two loads, a
// barrier); 37 int8 rows of 4096 -> 2047 11 (three 16-row tiles of x to each tile of weights, their sums through LDS).
// bfloat16 scales and biases take the same time as float16 ones (33 and 34 us, 6.3 and 6.4, 13.3 and 13.5 for bf16 rows).
//
// A workgroup's waves share K out (256 of it, a span, at a time) and keep their part of x in registers, so
// that x is read once a workgroup whatever the number of weight rows; their sums of some tiles of 16 weight
// rows are added through LDS between barriers that leave loads on their way.
#include "common.hpp"
#include "serve.hpp"

#pragma clang fp contract(off)

namespace moe {

namespace {

typedef __attribute__((__vector_size__(4 * sizeof(float)))) float f32x4;
typedef __attribute__((__vector_size__(8 * sizeof(_Float16)))) _Float16 f16x8;
typedef __attribute__((__vector_size__(4 * sizeof(int)))) int i32x4;


// Eight codes of a word as 16 + code, in the order 0 4 1 5 2 6 3 7.
template <LinX X>
__device__ __forceinline__ u32x4 codes_of(uint32_t w) {
  if constexpr (X == LinX::Bf16) {
    constexpr uint32_t m = 0x00780078u, o = 0x41804180u;
    return u32x4{(w << 3 & m) | o, (w >> 1 & m) | o, (w >> 5 & m) | o, (w >> 9 & m) | o};
  } else {
    constexpr uint32_t m = 0x03c003c0u, o = 0x4c004c00u;
    return u32x4{(w << 6 & m) | o, (w << 2 & m) | o, (w >> 2 & m) | o, (w >> 6 & m) | o};
  }
}
template <LinX X>
__device__ __forceinline__ f32x4 products(u32x4 a, u32x4 b, f32x4 c) {
  if constexpr (X == LinX::Bf16)
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
}
// Sixteen codes as bytes, in the order 0 2 4 6, 1 3 5 7, 8 10 12 14, 9 11 13 15.
__device__ __forceinline__ u32x4 bytes_of(uint2 w) {
  constexpr uint32_t m = 0x0f0f0f0fu;
  return u32x4{w.x & m, w.x >> 4 & m, w.y & m, w.y >> 4 & m};
}

// One group of 64 of 16 rows of x as matrix operands: lane (t, g) has row t's elements 16 g .. 16 g + 15 of the
// group, in the order of the codes' operands.  sum, scale: of rows 4 g + i (those of the lane's results).
template <LinX X>
struct Group {
  u32x4 x[X == LinX::Int8 ? 1 : 2];
  f32x4 sum, scale;
};
// t0: the first of the rows
template <LinX X>
__device__ __forceinline__ Group<X> load_group(const LinArgs &a, int64_t t0, int group) {
  const int lane = threadIdx.x & 63, g = lane >> 4;
  const int64_t t = t0 + (lane & 15);
  const bool in = t < a.T && group * 64 < a.k;
  const int64_t at = (in ? t * a.xld + group * 64 : 0) + 16 * g;
  Group<X> o;
  if constexpr (X == LinX::Int8) {
    u32x4 v = *(const u32x4 *)((const int8_t *)a.x + at);
    if (!in) v = u32x4{0, 0, 0, 0};
    o.x[0] = u32x4{__builtin_amdgcn_perm(v[1], v[0], 0x06040200u), __builtin_amdgcn_perm(v[1], v[0], 0x07050301u),
                   __builtin_amdgcn_perm(v[3], v[2], 0x06040200u), __builtin_amdgcn_perm(v[3], v[2], 0x07050301u)};
    constexpr int one = 0x01010101;
    const i32x4 s = __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(i32x4, o.x[0]), i32x4{one, one, one, one},
                                                          i32x4{0, 0, 0, 0}, 0, 0, 0);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int64_t r = t0 + 4 * g + i;
      o.sum[i] = (float)s[i];
      o.scale[i] = r < a.T && group * 64 < a.k ? a.xs[r * a.xs_cols + (a.xs_shift == 31 ? 0 : group >> a.xs_shift)] : 0.0f;
    }
  } else {
    o.sum = f32x4{0, 0, 0, 0};
    constexpr uint32_t one = X == LinX::Bf16 ? 0x3f803f80u : 0x3c003c00u;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      u32x4 v = *(const u32x4 *)((const uint16_t *)a.x + at + 8 * j);
      if (!in) v = u32x4{0, 0, 0, 0};
      pairs_p4(v[0], v[1], v[2], v[3], (uint32_t *)&o.x[j]);
      o.sum = products<X>(o.x[j], u32x4{one, one, one, one}, o.sum);
    }
  }
  return o;
}

// Weights of a tile of 16 rows and a span: lane (n, g) has row n's codes 16 g .. 16 g + 15 of each of its four
// groups, and the scale and bias of row n and group g.
struct Weights {
  uint2 code[4];
  uint16_t s, b;
};
__device__ __forceinline__ Weights load_weights(const LinArgs &a, int tile, int span, int ktiles) {
  const int lane = threadIdx.x & 63, n = lane & 15, g = lane >> 4;
  Weights w;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int kt = min(2 * span + i, ktiles - 1);  // (of a span that ends in its middle: the last one again)
    const uint32_t *c = a.codes + ((int64_t)tile * ktiles + kt) * 256 + n * 16 + 2 * g;
    w.code[2 * i] = *(const uint2 *)c;
    w.code[2 * i + 1] = *(const uint2 *)(c + 8);
  }
  const int64_t q = ((int64_t)tile * 2 * ktiles + min(4 * span + g, 2 * ktiles - 1)) * 16 + n;
  w.s = a.scale[q];
  w.b = a.bias[q];
  return w;
}

// acc[c] (rows 4 g + i of x, weight row n) += the products of one tile and span with 16 CT rows of x.
template <LinX X, int CT>
__device__ __forceinline__ void multiply(const Weights &w, const Group<X> (&x)[4][CT], bool qbf16, f32x4 (&acc)[CT]) {
  // the lane groups' scales and biases to all of them
  const uint32_t sb = (uint32_t)w.s | (uint32_t)w.b << 16;
  const auto h = __builtin_amdgcn_permlane32_swap(sb, sb, false, false);
  const auto lo = __builtin_amdgcn_permlane16_swap(h[0], h[0], false, false), hi = __builtin_amdgcn_permlane16_swap(h[1], h[1], false, false);
  const uint32_t q[4] = {lo[0], lo[1], hi[0], hi[1]};
#pragma unroll
  for (int gi = 0; gi < 4; ++gi) {
    const float s = qp_f32(q[gi] & 0xffffu, qbf16);
    float b = qp_f32(q[gi] >> 16, qbf16);
    if constexpr (X == LinX::Int8) {
      const u32x4 c = bytes_of(w.code[gi]);
#pragma unroll
      for (int t = 0; t < CT; ++t) {
        const i32x4 r = __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(i32x4, x[gi][t].x[0]), __builtin_bit_cast(i32x4, c),
                                                              i32x4{0, 0, 0, 0}, 0, 0, 0);
#pragma unroll
        for (int i = 0; i < 4; ++i)
          acc[t][i] = __builtin_fmaf(x[gi][t].scale[i], __builtin_fmaf(s, (float)r[i], b * x[gi][t].sum[i]), acc[t][i]);
      }
    } else {
      b = __builtin_fmaf(-16.0f, s, b);
      const u32x4 c0 = codes_of<X>(w.code[gi].x), c1 = codes_of<X>(w.code[gi].y);
#pragma unroll
      for (int t = 0; t < CT; ++t) {
        const f32x4 r = products<X>(x[gi][t].x[1], c1, products<X>(x[gi][t].x[0], c0, f32x4{0, 0, 0, 0}));
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[t][i] = __builtin_fmaf(s, r[i], __builtin_fmaf(b, x[gi][t].sum[i], acc[t][i]));
      }
    }
  }
}

__device__ __forceinline__ void store(const LinArgs &a, int64_t t, int n, float v) {
  const int64_t at = t * a.old + n;
  if (a.out_type == LinOut::Fp32) ((float *)a.out)[at] = v;
  else if (a.out_type == LinOut::Bf16) ((uint16_t *)a.out)[at] = f32_to_bf16(v);
  else ((_Float16 *)a.out)[at] = (_Float16)v;
}

// Barrier for LDS: loads from memory stay on their way.
__device__ __forceinline__ void lds_barrier() {
  asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// 16 CT rows of x, weight tiles in runs over the workgroups, R of them between barriers.  KS spans of K (w,
// w + waves, ...) are held by wave w for the whole run, and the weights of the next R tiles are on their way; KS 0: any
// number of spans, x read again for each weight tile.
template <LinX X, int CT, int KS, int R, int MAX_WAVES>
__global__ void __launch_bounds__(64 * MAX_WAVES) k_linear(LinArgs a) {
  extern __shared__ __align__(16) uint8_t lds_raw[];
  const int waves = blockDim.x >> 6, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int tiles = (a.n + 15) >> 4, ktiles = (a.k + 127) >> 7, spans = (ktiles + 1) >> 1;
  // The workgroups of one run of weight tiles, one for each 16 CT rows of x, follow each other at a distance of 8, so
  // that they run side by side on one XCD and its cache brings the weights once.  (Where there is a workgroup for each
  // tile, one after the other: 37 rows of 4096 -> 2047 11.3 us, 12.4 side by side.)
  const int id = blockIdx.x, cols = a.cols, runs = gridDim.x / cols;
  const int run = R == 1 ? id % runs : id / (8 * cols) * 8 + id % 8, col = R == 1 ? id / runs : id / 8 % cols;
  const int first = (int)((int64_t)tiles * run / runs), last = (int)((int64_t)tiles * (run + 1) / runs);
  if (first >= last) return;
  const int64_t t0 = (int64_t)col * 16 * CT;
  const int rows = (int)min((int64_t)16 * CT, a.T - t0);
  constexpr int kHeld = KS > 0 ? KS : 1;
  Group<X> x[kHeld][4][CT];
  auto load_x = [&](int span, Group<X> (&o)[4][CT]) {
#pragma unroll
    for (int gi = 0; gi < 4; ++gi)
#pragma unroll
      for (int c = 0; c < CT; ++c) o[gi][c] = load_group<X>(a, t0 + 16 * c, 4 * span + gi);
  };
  Weights w[R][kHeld];
  auto load = [&](int tile, Weights (&o)[kHeld]) {  // (the last one again behind the end: no branch)
#pragma unroll
    for (int i = 0; i < kHeld; ++i) o[i] = load_weights(a, min(tile, last - 1), min(wave + i * waves, spans - 1), ktiles);
  };
#pragma unroll
  for (int p = 0; p < R; ++p) load(first + p, w[p]);
  if constexpr (KS > 0) {
#pragma unroll
    for (int i = 0; i < KS; ++i) load_x(wave + i * waves, x[i]);  // (zeros behind the last span)
  }
  int buffer = 0;
  for (int tile = first; tile < last; tile += R) {
    f32x4 *red = (f32x4 *)lds_raw + buffer * waves * R * CT * 64;  // [waves][R][CT][64]
    buffer ^= 1;
#pragma unroll
    for (int p = 0; p < R; ++p) {
      f32x4 acc[CT];
#pragma unroll
      for (int c = 0; c < CT; ++c) acc[c] = f32x4{0, 0, 0, 0};
      if constexpr (KS > 0) {
#pragma unroll
        for (int i = 0; i < KS; ++i) multiply<X, CT>(w[p][i], x[i], a.qbf16, acc);
        load(tile + p + R, w[p]);
      } else {
        for (int span = wave; span < spans; span += waves) {
          load_x(span, x[0]);
          const Weights now = w[p][0];
          w[p][0] = load_weights(a, min(tile + p, last - 1), min(span + waves, spans - 1), ktiles);
          multiply<X, CT>(now, x[0], a.qbf16, acc);
        }
        w[p][0] = load_weights(a, min(tile + p + R, last - 1), min(wave, spans - 1), ktiles);
      }
#pragma unroll
      for (int c = 0; c < CT; ++c) red[((wave * R + p) * CT + c) * 64 + lane] = acc[c];
    }
    // (a buffer's next writes lie behind the next barrier, which no wave passes before all have read)
    lds_barrier();
    const int left = min(R, last - tile);
    for (int o = threadIdx.x; o < left * CT * 256; o += blockDim.x) {
      const int slot = o >> 8, t = o >> 4 & 15, n = o & 15;  // of [R][CT]
      const float *f = (const float *)(red + slot * 64) + ((t >> 2) * 16 + n) * 4 + (t & 3);
      float sum = 0.0f;
      float v[MAX_WAVES];
#pragma unroll
      for (int i = 0; i < MAX_WAVES; ++i) v[i] = i < waves ? f[i * R * CT * 256] : 0.0f;
#pragma unroll
      for (int i = 0; i < MAX_WAVES; ++i) sum += v[i];
      const int row = slot % CT * 16 + t, at = (tile + slot / CT) * 16 + n;
      if (row < rows && at < a.n) store(a, t0 + row, at, sum);
    }
  }
}

// per_cu: waves that a compute unit holds at once, by registers.
template <LinX X, int CT, int KS, int R, int MAX_WAVES>
hipError_t go(LinArgs a, int per_cu, hipStream_t s) {
  const int tiles = (a.n + 15) >> 4, spans = (a.k + 255) >> 8;
  const int waves = spans < MAX_WAVES ? spans : MAX_WAVES;
  const int64_t cols = (a.T + 16 * CT - 1) / (16 * CT);
  constexpr int kWaveLds = 2 * R * CT * 64 * 16;
  static_assert(kWaveLds * MAX_WAVES <= 160 * 1024, "two buffers");
  static std::atomic<uint64_t> done{0};
  const hipError_t e = allow_lds(k_linear<X, CT, KS, R, MAX_WAVES>, kWaveLds * MAX_WAVES, done);
  if (e != hipSuccess) return e;
  // runs of tiles that fill the chip once, or of R tiles; of one tile (a launch holds less than 2^32 work-items)
  int64_t runs = R == 1 ? (1 << 21) / cols : 256 * (per_cu / waves) / cols;
  if (runs > (tiles + R - 1) / R) runs = (tiles + R - 1) / R;
  if (runs < 1) runs = 1;
  if (cols > 1 && R > 1) runs = (runs + 7) / 8 * 8;
  a.cols = (int)cols;
  hipLaunchKernelGGL((k_linear<X, CT, KS, R, MAX_WAVES>), dim3((unsigned)(runs * cols)), dim3(64 * waves), kWaveLds * waves, s, a);
  return hipGetLastError();
}

template <LinX X>
hipError_t launch(const LinArgs &a, hipStream_t s) {
  const int64_t tiles = (a.n + 15) >> 4;
  const int spans = (a.k + 255) >> 8;
  // Up to 512 pairs of a weight tile and 16 rows of x: a workgroup for each, so that all compute units take part.
  // (us a call so and with runs: one row of 2048 -> 5120 6.2 and 8.2; 37 of 4096 -> 2047, int8, 11.3 and 16.2;
  // but 24 of 2048 -> 8192, 1024 pairs, 14.0 and 11.6, and 64 of 2048 -> 5120, 1280 pairs, 16.9 and 12.4.)
  if (tiles * ((a.T + 15) / 16) <= 512) {
    if (spans <= 8) return go<X, 1, 1, 1, 8>(a, 16, s);
    if (spans <= 16) return go<X, 1, 1, 1, 16>(a, 16, s);
    // (four spans of x held by a wave spill its registers: 8 rows of 8192 -> 8192 60 us, 22 read again)
    return go<X, 1, 0, 1, 16>(a, 16, s);
  }
  // 32 rows of x to a workgroup where their registers allow it.
  if (a.T > 16 && spans <= 8) return go<X, 2, 1, 4, 8>(a, 8, s);
  if (spans <= 8) return go<X, 1, 1, 4, 8>(a, 16, s);
  if (spans <= 16) return go<X, 1, 2, 4, 8>(a, 8, s);
  return go<X, 1, 0, 1, 16>(a, 16, s);
}

}  // namespace

hipError_t launch_linear(const LinArgs &a, hipStream_t s) {
  if (a.T <= 0) return hipSuccess;
  switch (a.x_type) {
    case LinX::Bf16: return launch<LinX::Bf16>(a, s);
    case LinX::Fp16: return launch<LinX::Fp16>(a, s);
    case LinX::Int8: return launch<LinX::Int8>(a, s);
  }
  return hipErrorInvalidValue;
}

}  // namespace moe
