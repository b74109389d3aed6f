// Products of few rows with 4-bit weights ("Optimizing on-device inference for Apple Silicon",
// section "Decode > Optimize the one-row weight path").
//
//     out[t][n] = sum_g s[n][g] (sum_{k in g} code x) + b[n][g] (sum_{k in g} x),  groups of 64.
//
// Bound: memory, 0.5625 bytes a weight, read once.  Even a single row goes over the matrix units:
// with weights as the row operand and the rows of x as the columns, 8 codes are turned into an operand's
// register with 8 vector instructions for up to 16 rows at once, where dot products need 4 more for
// each row.  Codes enter as 16 + code, which is exact in either type (the mantissa's top bits), so
// a group's products start from a sum of zero and are scaled in binary32:
//     acc += s r + (b - 16 s) X,   r = sum (16 + code) x,  X = sum x,
// where a larger offset (128 + code) would cost eight times the rounding.  int8 rows take the codes
// as bytes, and r and X are exact.
//
// A workgroup's waves share K out (128 of it at a time) and keep their part of x in registers, so
// that x is read once a workgroup whatever the number of weight rows; their sums of a tile of 16 weight
// rows are added through LDS by one wave while the others go on to the next tile.
#include "common.hpp"
#include "serve.hpp"

#pragma clang fp contract(off)

namespace moe {

namespace {

typedef __attribute__((__vector_size__(4 * sizeof(float)))) float f32x4;
typedef __attribute__((__vector_size__(8 * sizeof(_Float16)))) _Float16 f16x8;
typedef __attribute__((__vector_size__(4 * sizeof(int)))) int i32x4;

constexpr int kMaxWaves = 16;

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
// Sixteen codes as bytes, in the order 0 2 4 6, 1 3 5 7, 8 10 12 14, 9 11 13 15.
__device__ __forceinline__ u32x4 bytes_of(uint2 w) {
  constexpr uint32_t m = 0x0f0f0f0fu;
  return u32x4{w.x & m, w.x >> 4 & m, w.y & m, w.y >> 4 & m};
}

// Sum over the four 16-lane groups.
__device__ __forceinline__ float groups_sum(float v) {
  auto a = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  v = __uint_as_float(a[0]) + __uint_as_float(a[1]);
  auto b = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return __uint_as_float(b[0]) + __uint_as_float(b[1]);
}

// One group of 64 of up to 16 rows of x as matrix operands: lane (t, g) has row t's elements 16 g ..
// 16 g + 15 of the group, in the order of the codes' operands; the rows' sums, and int8 rows' scales.
template <LinX X>
struct Group {
  u32x4 x[X == LinX::Int8 ? 1 : 2];
  float sum, scale;
};
template <LinX X>
__device__ __forceinline__ Group<X> load_group(const LinArgs &a, int64_t t, int group) {
  const int g = (threadIdx.x & 63) >> 4;
  const bool in = t < a.T && group * 64 < a.k;
  const int64_t at = (in ? t * a.xld + group * 64 : 0) + 16 * g;
  Group<X> o;
  o.scale = 1.0f;
  if constexpr (X == LinX::Int8) {
    u32x4 v = *(const u32x4 *)((const int8_t *)a.x + at);
    if (!in) v = u32x4{0, 0, 0, 0};
    int s = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) s = __builtin_amdgcn_sdot4((int)v[i], 0x01010101, s, false);
    o.sum = groups_sum((float)s);
    o.x[0] = u32x4{__builtin_amdgcn_perm(v[1], v[0], 0x06040200u), __builtin_amdgcn_perm(v[1], v[0], 0x07050301u),
                   __builtin_amdgcn_perm(v[3], v[2], 0x06040200u), __builtin_amdgcn_perm(v[3], v[2], 0x07050301u)};
    o.scale = in ? a.xs[t * a.xs_cols + (a.xs_shift == 31 ? 0 : group >> a.xs_shift)] : 0.0f;
  } else {
    float s = 0.0f;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      u32x4 v = *(const u32x4 *)((const uint16_t *)a.x + at + 8 * j);
      if (!in) v = u32x4{0, 0, 0, 0};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if constexpr (X == LinX::Bf16) s += bf16_lo(v[i]) + bf16_hi(v[i]);
        else s += fp16_to_f32((uint16_t)v[i]) + fp16_to_f32((uint16_t)(v[i] >> 16));
      }
      pairs_p4(v[0], v[1], v[2], v[3], (uint32_t *)&o.x[j]);
    }
    o.sum = groups_sum(s);
  }
  return o;
}

// Weights of one tile of 16 rows and 128 k: lane (n, g) has row n's codes 16 g .. 16 g + 15 of both
// groups, and scales and biases of rows 4 g .. 4 g + 3, which are those of its results.
struct Weights {
  uint2 code[2], s[2], b[2];
};
__device__ __forceinline__ Weights load_weights(const LinArgs &a, int tile, int kt, int ktiles) {
  const int lane = threadIdx.x & 63, n = lane & 15, g = lane >> 4;
  Weights w;
  const uint32_t *c = a.codes + ((int64_t)tile * ktiles + kt) * 256 + n * 16 + 2 * g;
  const int64_t q = ((int64_t)tile * ktiles + kt) * 32 + 4 * g;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    w.code[i] = *(const uint2 *)(c + 8 * i);
    w.s[i] = *(const uint2 *)(a.scale + q + 16 * i);
    w.b[i] = *(const uint2 *)(a.bias + q + 16 * i);
  }
  return w;
}
__device__ __forceinline__ float qparam(uint2 w, int i, bool bf16) {
  const uint32_t v = i < 2 ? w.x : w.y;
  return qp_f32(i & 1 ? v >> 16 : v & 0xffffu, bf16);
}

// acc[c] (rows 4 g + i of the tile, row t of x) += the products of one tile with 16 CT rows of x.
template <LinX X, int CT>
__device__ __forceinline__ void multiply(const Weights &w, const Group<X> (&x)[2][CT], bool qbf16, f32x4 (&acc)[CT]) {
#pragma unroll
  for (int gi = 0; gi < 2; ++gi) {
    float s[4], b[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      s[i] = qparam(w.s[gi], i, qbf16);
      b[i] = qparam(w.b[gi], i, qbf16);
      if constexpr (X != LinX::Int8) b[i] = __builtin_fmaf(-16.0f, s[i], b[i]);
    }
    if constexpr (X == LinX::Int8) {
      const u32x4 c = bytes_of(w.code[gi]);
#pragma unroll
      for (int t = 0; t < CT; ++t) {
        const i32x4 r = __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(i32x4, c), __builtin_bit_cast(i32x4, x[gi][t].x[0]),
                                                              i32x4{0, 0, 0, 0}, 0, 0, 0);
#pragma unroll
        for (int i = 0; i < 4; ++i)
          acc[t][i] = __builtin_fmaf(x[gi][t].scale, __builtin_fmaf(s[i], (float)r[i], b[i] * x[gi][t].sum), acc[t][i]);
      }
    } else {
      const u32x4 c0 = codes_of<X>(w.code[gi].x), c1 = codes_of<X>(w.code[gi].y);
#pragma unroll
      for (int t = 0; t < CT; ++t) {
        f32x4 r = {0, 0, 0, 0};
        if constexpr (X == LinX::Bf16) {
          r = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, c0), __builtin_bit_cast(bf16x8, x[gi][t].x[0]), r, 0, 0, 0);
          r = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, c1), __builtin_bit_cast(bf16x8, x[gi][t].x[1]), r, 0, 0, 0);
        } else {
          r = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, c0), __builtin_bit_cast(f16x8, x[gi][t].x[0]), r, 0, 0, 0);
          r = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, c1), __builtin_bit_cast(f16x8, x[gi][t].x[1]), r, 0, 0, 0);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[t][i] = __builtin_fmaf(s[i], r[i], __builtin_fmaf(b[i], x[gi][t].sum, acc[t][i]));
      }
    }
  }
}

// Four results of row t, weight rows n0 .. n0 + 3.
__device__ __forceinline__ void store4(const LinArgs &a, int64_t t, int n0, f32x4 v) {
  if (t >= a.T) return;
  const int64_t at = t * a.old + n0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (n0 + i >= a.n) return;
    if (a.out_type == LinOut::Fp32) ((float *)a.out)[at + i] = v[i];
    else if (a.out_type == LinOut::Bf16) ((uint16_t *)a.out)[at + i] = f32_to_bf16(v[i]);
    else ((_Float16 *)a.out)[at + i] = (_Float16)v[i];
  }
}

// 16 CT rows of x, weight tiles in runs over the workgroups.  KW tiles of K (w, w + waves, ...) are
// held by wave w for the whole run; 0: any number, x read again for each weight tile.
template <LinX X, int CT, int KW>
__global__ void __launch_bounds__(64 * kMaxWaves) k_linear(LinArgs a) {
  extern __shared__ __align__(16) uint8_t lds_raw[];
  const int waves = blockDim.x >> 6, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  f32x4 *red = (f32x4 *)lds_raw;  // [2][waves][CT][64]
  const int tiles = (a.n + 15) >> 4, ktiles = (a.k + 127) >> 7;
  const int first = (int)((int64_t)tiles * blockIdx.x / gridDim.x), last = (int)((int64_t)tiles * (blockIdx.x + 1) / gridDim.x);
  const int64_t t0 = (int64_t)blockIdx.y * 16 * CT;
  constexpr int kHeld = KW > 0 ? KW : 1;
  Weights w[kHeld];
  Group<X> x[kHeld][2][CT];
  auto load_x = [&](int kt, Group<X> (&o)[2][CT]) {
#pragma unroll
    for (int gi = 0; gi < 2; ++gi)
#pragma unroll
      for (int c = 0; c < CT; ++c) o[gi][c] = load_group<X>(a, t0 + 16 * c + (lane & 15), 2 * kt + gi);
  };
  if constexpr (KW > 0) {
#pragma unroll
    for (int i = 0; i < KW; ++i)
      if (first < last) w[i] = load_weights(a, first, min(wave + i * waves, ktiles - 1), ktiles);
#pragma unroll
    for (int i = 0; i < KW; ++i) load_x(wave + i * waves, x[i]);  // (zeros behind the last tile)
  }
  for (int tile = first; tile < last; ++tile) {
    f32x4 acc[CT];
#pragma unroll
    for (int c = 0; c < CT; ++c) acc[c] = f32x4{0, 0, 0, 0};
    if constexpr (KW > 0) {
      Weights now[KW];
#pragma unroll
      for (int i = 0; i < KW; ++i) {
        now[i] = w[i];
        if (tile + 1 < last) w[i] = load_weights(a, tile + 1, min(wave + i * waves, ktiles - 1), ktiles);
      }
#pragma unroll
      for (int i = 0; i < KW; ++i) multiply<X, CT>(now[i], x[i], a.qbf16, acc);
    } else {
      for (int kt = wave; kt < ktiles; kt += waves) {
        w[0] = load_weights(a, tile, kt, ktiles);
        load_x(kt, x[0]);
        multiply<X, CT>(w[0], x[0], a.qbf16, acc);
      }
    }
    if (waves > 1) {
      f32x4 *mine = red + (tile & 1) * waves * CT * 64;
#pragma unroll
      for (int c = 0; c < CT; ++c) mine[(wave * CT + c) * 64 + lane] = acc[c];
      __syncthreads();
      // one wave adds, another one each time; its reads are done before it reaches the next
      // barrier, behind which this buffer's next writes lie
      if (wave != (tile - first) % waves) continue;
#pragma unroll
      for (int c = 0; c < CT; ++c) {
        acc[c] = mine[c * 64 + lane];
        for (int v = 1; v < waves; ++v) acc[c] += mine[(v * CT + c) * 64 + lane];
      }
    }
#pragma unroll
    for (int c = 0; c < CT; ++c) store4(a, t0 + 16 * c + (lane & 15), tile * 16 + 4 * (lane >> 4), acc[c]);
  }
}

template <LinX X, int CT, int KW>
hipError_t go(const LinArgs &a, int waves, hipStream_t s) {
  const int tiles = (a.n + 15) >> 4;
  const int64_t cols = (a.T + 16 * CT - 1) / (16 * CT);
  const int lds = waves > 1 ? 2 * waves * CT * 64 * 16 : 0;
  static std::atomic<uint64_t> done{0};
  const hipError_t e = allow_lds(k_linear<X, CT, KW>, 2 * kMaxWaves * CT * 64 * 16, done);
  if (e != hipSuccess) return e;
  const int most = 256 * (kMaxWaves / waves);
  hipLaunchKernelGGL((k_linear<X, CT, KW>), dim3(tiles < most ? tiles : most, (unsigned)cols), dim3(64 * waves), lds, s, a);
  return hipGetLastError();
}

template <LinX X>
hipError_t launch(const LinArgs &a, hipStream_t s) {
  const int ktiles = (a.k + 127) >> 7;
  const int waves = ktiles < kMaxWaves ? ktiles : kMaxWaves;
  const int held = (ktiles + waves - 1) / waves;
  if (a.T <= 16) return held == 1 ? go<X, 1, 1>(a, waves, s) : held == 2 ? go<X, 1, 2>(a, waves, s) : go<X, 1, 0>(a, waves, s);
  if (a.T <= 32) return held == 1 ? go<X, 2, 1>(a, waves, s) : go<X, 2, 0>(a, waves, s);
  return held == 1 ? go<X, 4, 1>(a, waves, s) : go<X, 4, 0>(a, waves, s);
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
