// Root-mean-square norm with the residual's addition, and an output in 8 bits with scales.
//
// Per row: h = x + r, y = h (mean(h^2) + eps)^(-1/2) (offset + w), and in 8 bits s = max|y| / 127
// (448), code = y / s rounded.  Every element is read once, held in registers as binary32 while
// the row's sum goes round, and written once.
//
// A row of more than 1024 elements lies over a workgroup, 8 elements a lane at 2048: 4 rows of
// 2048 2.45 us (a row on one wave: 3.9) and 8192 of them 24 us (29).  Shorter rows take the lanes
// they fill, down to 8.
//
// Bound: the launch for few rows (2.5 us), memory for many: 8192 rows of 2048 bf16, residual and
// both outputs 24 us (5.6 TB/s), with int8 or e4m3 in groups of 128 22.5 to 24.5 us (4.8 TB/s); 24496 heads of 256
// fp16 out of rows of 20 7.7 us (3.3 TB/s: 1/5 of each row is passed over).  Stores that go round
// the caches take 10% off a large norm alone and cost the product that reads it next more
// (8192 rows, norm, product and norm 260 -> 263 us), so they are ordinary ones.  Weights loaded
// ahead of the row's sum changed nothing for few rows and cost many 1.5 us.
#include "common.hpp"
#include "serve.hpp"

#pragma clang fp contract(off)

namespace moe {

namespace {

constexpr int kThreads = 256;

template <bool F16>
__device__ __forceinline__ float value(uint32_t w) {
  return F16 ? fp16_to_f32((uint16_t)w) : bf16_to_f32((uint16_t)w);
}
template <bool F16>
__device__ __forceinline__ uint32_t pair_of(float lo, float hi) {
  if constexpr (F16) {
    typedef __attribute__((__vector_size__(2 * sizeof(_Float16)))) _Float16 f16x2;
    return __builtin_bit_cast(uint32_t, f16x2{(_Float16)lo, (_Float16)hi});
  } else {
    return pack_bf16x2(lo, hi);
  }
}

// Over the LANES consecutive lanes that hold a row (every lane gets the result).
template <int LANES>
__device__ __forceinline__ float lanes_sum(float v) {
  if constexpr (LANES >= 64) return wave_sum(v);
  if constexpr (LANES == 8) {
    v += dpp_f<0xB1>(v);   // quad_perm [1,0,3,2]
    v += dpp_f<0x4E>(v);   // quad_perm [2,3,0,1]
    v += dpp_f<0x141>(v);  // row_half_mirror
    return v;
  }
  v = row16_sum(v);
  if constexpr (LANES == 32) {
    auto a = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = __uint_as_float(a[0]) + __uint_as_float(a[1]);
  }
  return v;
}
// Maximum of bit patterns of magnitudes, whose order puts NaN above infinity above numbers.
template <int C>
__device__ __forceinline__ uint32_t dpp_max(uint32_t v) {
  return max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, C, 0xf, 0xf, false));
}
template <int LANES>
__device__ __forceinline__ uint32_t lanes_max(uint32_t v) {
  if constexpr (LANES >= 64) return wave_max_u32(v);
  v = dpp_max<0xB1>(v);
  v = dpp_max<0x4E>(v);
  if constexpr (LANES >= 8) v = dpp_max<0x141>(v);  // row_half_mirror
  if constexpr (LANES >= 16) v = dpp_max<0x140>(v);  // row_mirror
  if constexpr (LANES == 32) {
    auto a = __builtin_amdgcn_permlane16_swap(v, v, false, false);
    v = max(a[0], a[1]);
  }
  return v;
}

// Scale of a group whose largest magnitude has these bits, and what its elements are multiplied by
// to get codes (e4m3: to get half of them, for 448 / 2^-120 would overflow).
struct Step {
  float scale, inv;
};
template <int KIND>
__device__ __forceinline__ Step step_of(uint32_t top) {
  constexpr float kMost = KIND == 1 ? 127.0f : 448.0f, kInv = KIND == 1 ? 127.0f : 224.0f;
  const float t = __uint_as_float(top);
  if (!(t < INFINITY)) return Step{t, 0.0f};
  if (t < 0x1p-120f) return Step{0.0f, 0.0f};  // (127 / t and 224 / t would overflow)
  return Step{t / kMost, kInv / t};
}
template <int KIND>
__device__ __forceinline__ float code_of(float y, const Step &s) {
  constexpr float kMost = KIND == 1 ? 127.0f : 448.0f;
  float c = s.inv == 0.0f ? 0.0f : y * s.inv;
  if constexpr (KIND == 2) c += c;
  return fminf(fmaxf(c, -kMost), kMost);
}
// Four codes packed into a word.
template <int KIND>
__device__ __forceinline__ uint32_t codes4(const float *y, const Step &s) {
  if constexpr (KIND == 1) {
    uint32_t w = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) w |= ((uint32_t)(int)__builtin_rintf(code_of<KIND>(y[i], s)) & 0xffu) << (8 * i);
    return w;
  } else {
    int w = __builtin_amdgcn_cvt_pk_fp8_f32(code_of<KIND>(y[0], s), code_of<KIND>(y[1], s), 0, false);
    return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(code_of<KIND>(y[2], s), code_of<KIND>(y[3], s), w, true);
  }
}
// Element offset of row `row` of an array.
__device__ __forceinline__ int64_t place(const Rows &a, int64_t t, int h) { return t * a.ts + h * a.hs; }

// Elements are handled eight at a time.  WIDE: all arrays and rows are aligned for that and rows hold whole
// eights.  Otherwise the same accesses are made at addresses aligned to an element (4271 rows of 3326 bf16,
// residual and both outputs, 28 us; one element at a time 82), and a row's last elements one by one.
typedef u32x4 __attribute__((aligned(2))) u32x4_2;
typedef uint32_t __attribute__((__vector_size__(2 * sizeof(uint32_t)), aligned(1))) u32x2_1;
template <class F>
__device__ __forceinline__ void last_ones(int at, int W, F f) {
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (at + i < W) f(i);
}
template <bool WIDE>
__device__ __forceinline__ u32x4 load8(const uint16_t *p, int at, int W) {
  if constexpr (WIDE) return *(const u32x4 *)(p + at);
  if (at + 8 <= W) return *(const u32x4_2 *)(p + at);
  u32x4 v = {0, 0, 0, 0};
  last_ones(at, W, [&](int i) { v[i / 2] |= (uint32_t)p[at + i] << (16 * (i % 2)); });
  return v;
}
// x + r, 0 behind the row's end
template <bool F16, bool WIDE>
__device__ __forceinline__ void load_h(const uint16_t *x, const uint16_t *r, int at, int W, float *h) {
  const u32x4 a = load8<WIDE>(x, at, W);
  u32x4 b = {0, 0, 0, 0};
  if (r) b = load8<WIDE>(r, at, W);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    h[2 * i] = value<F16>(a[i] & 0xffffu);
    h[2 * i + 1] = value<F16>(a[i] >> 16);
    if (r) {
      h[2 * i] += value<F16>(b[i] & 0xffffu);
      h[2 * i + 1] += value<F16>(b[i] >> 16);
    }
  }
}
template <bool F16, bool WIDE>
__device__ __forceinline__ void store_h(uint16_t *o, int at, int W, const float *h) {
  const u32x4 v = {pair_of<F16>(h[0], h[1]), pair_of<F16>(h[2], h[3]), pair_of<F16>(h[4], h[5]), pair_of<F16>(h[6], h[7])};
  if constexpr (WIDE) {
    *(u32x4 *)(o + at) = v;
  } else {
    if (at + 8 <= W) *(u32x4_2 *)(o + at) = v;
    else last_ones(at, W, [&](int i) { o[at + i] = (uint16_t)(v[i / 2] >> (16 * (i % 2))); });
  }
}
template <bool F16, bool WIDE>
__device__ __forceinline__ void load_w(const uint16_t *w, float offset, int at, int W, float *o) {
#pragma unroll
  for (int i = 0; i < 8; ++i) o[i] = offset;
  if (!w) return;
  const u32x4 a = load8<WIDE>(w, at, W);
#pragma unroll
  for (int i = 0; i < 8; ++i) o[i] += value<F16>(i & 1 ? a[i / 2] >> 16 : a[i / 2] & 0xffffu);
}
template <int KIND, bool WIDE>
__device__ __forceinline__ void store_codes(uint8_t *o, int at, int W, const float *y, const Step &s) {
  const uint32_t lo = codes4<KIND>(y, s), hi = codes4<KIND>(y + 4, s);
  if constexpr (WIDE) {
    *(uint2 *)(o + at) = make_uint2(lo, hi);
  } else {
    if (at + 8 <= W) *(u32x2_1 *)(o + at) = u32x2_1{lo, hi};
    else last_ones(at, W, [&](int i) { o[at + i] = (uint8_t)((i < 4 ? lo : hi) >> (8 * (i % 4))); });
  }
}

__device__ __forceinline__ uint32_t bits_of(float y) { return __float_as_uint(y) & 0x7fffffffu; }

// Of a group of `group` elements that lies over consecutive lanes, 8 elements each.
__device__ __forceinline__ uint32_t group_max(uint32_t v, int group) {
  return group == 64 ? lanes_max<8>(v) : group == 32 ? lanes_max<4>(v) : lanes_max<16>(v);
}

// A launch holds less than 2^32 work-items along x, so the workgroups of many rows lie over y as well.
constexpr int64_t kGridX = 1 << 20;
__device__ __forceinline__ int64_t block_of() { return (int64_t)blockIdx.y * gridDim.x + blockIdx.x; }
dim3 grid_of(int64_t blocks) {
  return blocks <= kGridX ? dim3((unsigned)blocks) : dim3((unsigned)kGridX, (unsigned)((blocks + kGridX - 1) / kGridX));
}

// A row over LANES lanes (256: a whole workgroup), 8 NV elements each: LANES * 8 NV >= W.
template <bool F16, int KIND, bool WIDE, int LANES, int NV>
__global__ void __launch_bounds__(kThreads) k_norm(NormArgs a) {
  __shared__ float red[4];
  __shared__ uint32_t redm[4];
  constexpr int kRows = kThreads / LANES;
  const int tid = threadIdx.x, lane = tid % LANES;
  const int64_t row = block_of() * kRows + tid / LANES;
  const bool live = row < a.rows;
  const int64_t rr = live ? row : a.rows - 1;
  const int64_t t = a.n == 1 ? rr : rr / a.n;
  const int hd = a.n == 1 ? 0 : (int)(rr - t * a.n);
  const uint16_t *x = (const uint16_t *)a.x.p + place(a.x, t, hd);
  const uint16_t *r = a.r.p ? (const uint16_t *)a.r.p + place(a.r, t, hd) : nullptr;
  float h[NV][8];
  float ss = 0.0f;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int at = (i * LANES + lane) * 8;
    if (at < a.W) {
      load_h<F16, WIDE>(x, r, at, a.W, h[i]);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) h[i][e] = 0.0f;
    }
  }
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int e = 0; e < 8; ++e) ss = __builtin_fmaf(h[i][e], h[i][e], ss);
  ss = lanes_sum<LANES>(ss);
  if constexpr (LANES == kThreads) {
    if ((tid & 63) == 0) red[tid >> 6] = ss;
    __syncthreads();
    ss = (red[0] + red[1]) + (red[2] + red[3]);
  }
  const float f = 1.0f / __builtin_sqrtf(ss / (float)a.W + a.eps);
  uint16_t *sum = a.sum.p ? (uint16_t *)a.sum.p + place(a.sum, t, hd) : nullptr;
  const int64_t out = place(a.out, t, hd);
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int at = (i * LANES + lane) * 8;
    if (at >= a.W) continue;
    if (sum && live) store_h<F16, WIDE>(sum, at, a.W, h[i]);
    float w[8];
    load_w<F16, WIDE>(a.w, a.offset, at, a.W, w);
#pragma unroll
    for (int e = 0; e < 8; ++e) h[i][e] = h[i][e] * f * w[e];
    if constexpr (KIND == 0) {
      if (live) store_h<F16, WIDE>((uint16_t *)a.out.p + out, at, a.W, h[i]);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) top = max(top, bits_of(h[i][e]));
    }
  }
  if constexpr (KIND > 0) {
    uint8_t *o = (uint8_t *)a.out.p + out;
    if (a.group == a.W) {
      top = lanes_max<LANES>(top);
      if constexpr (LANES == kThreads) {
        if ((tid & 63) == 0) redm[tid >> 6] = top;
        __syncthreads();
        top = max(max(redm[0], redm[1]), max(redm[2], redm[3]));
      }
      const Step s = step_of<KIND>(top);
      if (live && lane == 0) a.scale[rr] = s.scale;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int at = (i * LANES + lane) * 8;
        if (at < a.W && live) store_codes<KIND, WIDE>(o, at, a.W, h[i], s);
      }
    } else if constexpr (WIDE) {
      const int groups = a.W / a.group;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int at = (i * LANES + lane) * 8;
        uint32_t m = 0;  // (a lane behind the row's end is in no group of one before it)
        if (at < a.W) {
#pragma unroll
          for (int e = 0; e < 8; ++e) m = max(m, bits_of(h[i][e]));
        }
        const Step s = step_of<KIND>(group_max(m, a.group));
        if (at >= a.W || !live) continue;
        if (at % a.group == 0) a.scale[rr * groups + at / a.group] = s.scale;
        store_codes<KIND, WIDE>(o, at, a.W, h[i], s);
      }
    }
  }
}

// Rows too long for registers, one a workgroup: h is formed anew in each pass and written in the
// last, so that it may be written over what it comes from.  Bound: memory for many rows (1000 of 32768
// bf16, no residual, 31.5 us, 131 MB; int8 with one scale a row, a third pass, 44.5), a workgroup's own reads for few (64
// of 65536 27 us, 8 of 2^20 486: the other compute units have nothing to do).
template <bool F16, int KIND, bool WIDE>
__global__ void __launch_bounds__(kThreads) k_norm_long(NormArgs a) {
  __shared__ float red[4];
  __shared__ uint32_t redm[4];
  const int tid = threadIdx.x;
  const int64_t row = block_of(), t = row / a.n;
  if (row >= a.rows) return;
  const int hd = (int)(row - t * a.n);
  const uint16_t *x = (const uint16_t *)a.x.p + place(a.x, t, hd);
  const uint16_t *r = a.r.p ? (const uint16_t *)a.r.p + place(a.r, t, hd) : nullptr;
  float ss = 0.0f;
  for (int at = tid * 8; at < a.W; at += kThreads * 8) {
    float h[8];
    load_h<F16, WIDE>(x, r, at, a.W, h);
#pragma unroll
    for (int e = 0; e < 8; ++e) ss = __builtin_fmaf(h[e], h[e], ss);
  }
  ss = wave_sum(ss);
  if ((tid & 63) == 0) red[tid >> 6] = ss;
  __syncthreads();
  ss = (red[0] + red[1]) + (red[2] + red[3]);
  const float f = 1.0f / __builtin_sqrtf(ss / (float)a.W + a.eps);
  auto normed = [&](int at, float *h, float *y) {
    float w[8];
    load_h<F16, WIDE>(x, r, at, a.W, h);
    load_w<F16, WIDE>(a.w, a.offset, at, a.W, w);
#pragma unroll
    for (int e = 0; e < 8; ++e) y[e] = h[e] * f * w[e];
  };
  Step s{};
  if (KIND > 0 && a.group == a.W) {
    uint32_t top = 0;
    for (int at = tid * 8; at < a.W; at += kThreads * 8) {
      float h[8], y[8];
      normed(at, h, y);
#pragma unroll
      for (int e = 0; e < 8; ++e) top = max(top, bits_of(y[e]));
    }
    top = wave_max_u32(top);
    if ((tid & 63) == 0) redm[tid >> 6] = top;
    __syncthreads();
    s = step_of<KIND>(max(max(redm[0], redm[1]), max(redm[2], redm[3])));
    if (tid == 0) a.scale[row] = s.scale;
  }
  uint16_t *sum = a.sum.p ? (uint16_t *)a.sum.p + place(a.sum, t, hd) : nullptr;
  const int64_t out = place(a.out, t, hd);
  for (int b = 0; b < a.W; b += kThreads * 8) {
    const int at = b + tid * 8;
    const bool in = at < a.W;
    float h[8], y[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) y[e] = 0.0f;
    if (in) normed(at, h, y);
    if constexpr (KIND > 0 && WIDE) {
      if (a.group != a.W) {
        uint32_t m = 0;
#pragma unroll
        for (int e = 0; e < 8; ++e) m = max(m, bits_of(y[e]));
        s = step_of<KIND>(group_max(m, a.group));
        if (in && at % a.group == 0) a.scale[row * (a.W / a.group) + at / a.group] = s.scale;
      }
    }
    if (!in) continue;
    if (sum) store_h<F16, WIDE>(sum, at, a.W, h);
    if constexpr (KIND == 0)
      store_h<F16, WIDE>((uint16_t *)a.out.p + out, at, a.W, y);
    else
      store_codes<KIND, WIDE>((uint8_t *)a.out.p + out, at, a.W, y, s);
  }
}

template <bool F16, int KIND, bool WIDE, int LANES, int NV>
hipError_t go(const NormArgs &a, hipStream_t s) {
  constexpr int kRows = kThreads / LANES;
  hipLaunchKernelGGL((k_norm<F16, KIND, WIDE, LANES, NV>), grid_of((a.rows + kRows - 1) / kRows), dim3(kThreads), 0, s, a);
  return hipGetLastError();
}

template <bool F16, int KIND, bool WIDE>
hipError_t launch(const NormArgs &a, hipStream_t s) {
  if (a.W > 16384) {
    hipLaunchKernelGGL((k_norm_long<F16, KIND, WIDE>), grid_of(a.rows), dim3(kThreads), 0, s, a);
    return hipGetLastError();
  }
  // (groups of 128 elements lie over 16 lanes)
  if (a.W <= 64 && (KIND == 0 || a.group <= 64)) return go<F16, KIND, WIDE, 8, 1>(a, s);
  if (a.W <= 128) return go<F16, KIND, WIDE, 16, 1>(a, s);
  if (a.W <= 256) return go<F16, KIND, WIDE, 32, 1>(a, s);
  if (a.W <= 512) return go<F16, KIND, WIDE, 64, 1>(a, s);
  if (a.W <= 1024) return go<F16, KIND, WIDE, 64, 2>(a, s);
  if (a.W <= 2048) return go<F16, KIND, WIDE, 256, 1>(a, s);
  if (a.W <= 4096) return go<F16, KIND, WIDE, 256, 2>(a, s);
  if (a.W <= 8192) return go<F16, KIND, WIDE, 256, 4>(a, s);
  return go<F16, KIND, WIDE, 256, 8>(a, s);
}
template <bool F16, int KIND>
hipError_t launch(const NormArgs &a, hipStream_t s) {
  return a.vec ? launch<F16, KIND, true>(a, s) : launch<F16, KIND, false>(a, s);
}

}  // namespace

hipError_t launch_rms_norm(const NormArgs &a, hipStream_t s) {
  if (a.rows <= 0) return hipSuccess;
  switch (2 * a.out_kind + (a.fp16 ? 1 : 0)) {
    case 0: return launch<false, 0>(a, s);
    case 1: return launch<true, 0>(a, s);
    case 2: return launch<false, 1>(a, s);
    case 3: return launch<true, 1>(a, s);
    case 4: return launch<false, 2>(a, s);
    case 5: return launch<true, 2>(a, s);
  }
  return hipErrorInvalidValue;
}

}  // namespace moe
