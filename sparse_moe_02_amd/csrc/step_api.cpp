// Host side of the C ABI declared in include/norm.h, include/linear.h and include/sample.h: argument checks and
// launches.  Every check precedes every launch.
#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdint>

#include "../../include/linear.h"
#include "../../include/norm.h"
#include "../../include/sample.h"
#include "checks.hpp"

using namespace moe;

namespace {

// Strides and address of an array of `size`-byte elements.
moe_status check_rows(const moe_heads *x, int size) {
  if (!x || !x->p) return MOE_ERR_NULL;
  if (!aligned(x->p, size)) return MOE_ERR_ALIGN;
  if (x->token_stride < 0 || x->head_stride < 0 || x->token_stride > int64_t(1) << 38 ||
      x->head_stride > int64_t(1) << 38)
    return MOE_ERR_SHAPE;
  return MOE_OK;
}
bool wide(const moe_heads &x, int bytes) {
  return aligned(x.p, bytes) && x.token_stride % 8 == 0 && x.head_stride % 8 == 0;
}
bool same(const moe_heads &a, const moe_heads &b) {
  return a.p == b.p && a.token_stride == b.token_stride && a.head_stride == b.head_stride;
}
Rows dev_rows(const moe_heads *x) {
  return x ? Rows{const_cast<void *>(x->p), x->token_stride, x->head_stride} : Rows{};
}

// Places of moe_sample's arrays in its workspace.
struct SampleWs {
  int chunks, room;
  size_t mass, count, row, kept, list, total;
};
SampleWs sample_ws(int64_t R, int32_t V) {
  auto up = [](size_t n) { return (n + 255) & ~size_t(255); };
  SampleWs w;
  w.chunks = (V + 7 + kSampleChunk - 1) / kSampleChunk;  // (a row may start up to 7 elements behind a 16-byte block)
  w.room = V < kSampleList ? V : kSampleList;
  const size_t n = (size_t)R * w.chunks;
  w.mass = up(n * sizeof(SampleChunk));
  w.count = w.mass + up(n * kSampleBins * 8);
  w.row = w.count + up(n * kSampleBins * 4);
  w.kept = w.row + up((size_t)R * sizeof(SampleRow));
  w.list = w.kept + up(n * 8);
  w.total = w.list + (size_t)R * w.room * 8;
  return w;
}

}  // namespace

extern "C" {

moe_status moe_rms_norm(int64_t T, int32_t n_heads, int32_t width, moe_dtype dtype, const moe_heads *x,
                        const moe_heads *residual, const moe_heads *sum, const void *weight, float offset, float eps,
                        moe_dtype out_dtype, const moe_heads *out, int32_t group, float *scale, hipStream_t stream) {
  if (T < 0 || T > kMaxTokens) return MOE_ERR_TOKENS;
  if (n_heads < 1 || n_heads > 4096 || width < 1 || width > 1 << 20) return MOE_ERR_SHAPE;
  if (T * n_heads > int64_t(1) << 28) return MOE_ERR_TOKENS;
  if (dtype != MOE_BF16 && dtype != MOE_FP16) return MOE_ERR_DTYPE;
  if (out_dtype != dtype && out_dtype != MOE_INT8 && out_dtype != MOE_FP8) return MOE_ERR_DTYPE;
  const bool codes = out_dtype != dtype;
  if (!(eps >= 0.0f) || !std::isfinite(eps) || !std::isfinite(offset)) return MOE_ERR_SHAPE;
  if (group != 0 && (!codes || (group != 32 && group != 64 && group != 128) || width % group)) return MOE_ERR_SHAPE;
  if (T == 0) return MOE_OK;
  if (codes != (scale != nullptr)) return MOE_ERR_NULL;
  moe_status st = check_rows(x, 2);
  if (st != MOE_OK || (st = check_rows(out, codes ? 1 : 2)) != MOE_OK) return st;
  if (residual && (st = check_rows(residual, 2)) != MOE_OK) return st;
  if (sum && (st = check_rows(sum, 2)) != MOE_OK) return st;
  if (!aligned(weight, 2) || !aligned(scale, 4)) return MOE_ERR_ALIGN;
  if (!heads_distinct(*out, T, n_heads, width) || (sum && !heads_distinct(*sum, T, n_heads, width))) return MOE_ERR_SHAPE;
  const bool vec = width % 8 == 0 && wide(*x, 16) && (!residual || wide(*residual, 16)) && (!sum || wide(*sum, 16)) &&
                   wide(*out, codes ? 8 : 16) && aligned(weight, 16);
  if (group != 0 && !vec) return MOE_ERR_ALIGN;
  const int64_t W = width;
  const Span ss{scale, 4 * (uint64_t)(T * n_heads) * (uint64_t)(group ? width / group : 1)}, sw{weight, 2 * (uint64_t)W};
  const Span so{out->p, (uint64_t)(((T - 1) * out->token_stride + (n_heads - 1) * out->head_stride + W) * (codes ? 1 : 2))};
  const Span sh = sum ? span(*sum, T, n_heads, W) : Span{}, sx = span(*x, T, n_heads, W);
  const Span sr = residual ? span(*residual, T, n_heads, W) : Span{};
  for (const Span &w : {so, sh, ss})
    if (overlap(w, sw)) return MOE_ERR_ALIAS;
  for (const Span &o : {sx, sr, sh, so})
    if (overlap(ss, o)) return MOE_ERR_ALIAS;
  for (const moe_heads *r : {x, residual}) {
    if (!r) continue;
    if (sum && !same(*sum, *r) && heads_overlap(*sum, n_heads, *r, n_heads, T, W)) return MOE_ERR_ALIAS;
    if (codes ? overlap(so, span(*r, T, n_heads, W)) : !same(*out, *r) && heads_overlap(*out, n_heads, *r, n_heads, T, W))
      return MOE_ERR_ALIAS;
  }
  if (sum && (codes ? overlap(so, sh) : heads_overlap(*out, n_heads, *sum, n_heads, T, W))) return MOE_ERR_ALIAS;
  if ((st = device_ok()) != MOE_OK) return st;
  NormArgs a{};
  a.x = dev_rows(x);
  a.r = dev_rows(residual);
  a.sum = dev_rows(sum);
  a.out = dev_rows(out);
  a.w = static_cast<const uint16_t *>(weight);
  a.scale = scale;
  a.rows = T * n_heads;
  a.n = n_heads;
  a.W = width;
  a.group = group ? group : width;
  a.offset = offset;
  a.eps = eps;
  a.out_kind = !codes ? 0 : out_dtype == MOE_INT8 ? 1 : 2;
  a.fp16 = dtype == MOE_FP16;
  a.vec = vec;
  return launch_rms_norm(a, stream) == hipSuccess ? MOE_OK : MOE_ERR_HIP;
}

moe_status moe_linear(const moe_linear_weights *w, int64_t T, const void *x, int64_t x_stride, moe_dtype x_dtype,
                      const float *x_scale, int32_t x_group, void *out, int64_t out_stride, moe_dtype out_dtype,
                      hipStream_t stream) {
  if (!w) return MOE_ERR_NULL;
  if (w->n < 1 || w->n > 1 << 24 || w->k < 64 || w->k > 1 << 17 || w->k % 64) return MOE_ERR_SHAPE;
  if (w->qparam_dtype != MOE_FP16 && w->qparam_dtype != MOE_BF16) return MOE_ERR_DTYPE;
  if (x_dtype != MOE_BF16 && x_dtype != MOE_FP16 && x_dtype != MOE_INT8) return MOE_ERR_DTYPE;
  if (out_dtype != MOE_BF16 && out_dtype != MOE_FP16 && out_dtype != MOE_FP32) return MOE_ERR_DTYPE;
  if (T < 0 || T > kMaxTokens || T * w->n > int64_t(1) << 40) return MOE_ERR_TOKENS;
  const bool int8 = x_dtype == MOE_INT8;
  if (x_group != 0 && (!int8 || (x_group != 64 && x_group != 128) || w->k % x_group)) return MOE_ERR_SHAPE;
  const int64_t xe = int8 ? 1 : 2, oe = out_dtype == MOE_FP32 ? 4 : 2;
  if (x_stride < 0 || x_stride > int64_t(1) << 38 || out_stride > int64_t(1) << 38) return MOE_ERR_SHAPE;
  if (T > 1 && out_stride < w->n) return MOE_ERR_SHAPE;
  if (!w->codes || !w->scale || !w->bias) return MOE_ERR_NULL;
  if (!aligned(w->codes, 16) || !aligned(w->scale, 16) || !aligned(w->bias, 16)) return MOE_ERR_ALIGN;
  if (T == 0) return MOE_OK;
  if (!x || !out || int8 != (x_scale != nullptr)) return MOE_ERR_NULL;
  if (!aligned(x, 16) || x_stride * xe % 16 || !aligned(x_scale, 4) || !aligned(out, oe)) return MOE_ERR_ALIGN;
  const uint64_t rows = ((uint64_t)w->n + 15) / 16 * 16, kp = ((uint64_t)w->k + 127) / 128 * 128;
  const int cols = !int8 ? 0 : x_group ? w->k / x_group : 1;
  const Span so{out, (uint64_t)(((T - 1) * out_stride + w->n) * oe)};
  for (const Span &r : {Span{x, (uint64_t)(((T - 1) * x_stride + w->k) * xe)}, Span{x_scale, 4 * (uint64_t)T * cols},
                        Span{w->codes, rows * kp / 2}, Span{w->scale, rows * kp / 32}, Span{w->bias, rows * kp / 32}})
    if (overlap(so, r)) return MOE_ERR_ALIAS;
  const moe_status st = device_ok();
  if (st != MOE_OK) return st;
  LinArgs a{};
  a.codes = w->codes;
  a.scale = static_cast<const uint16_t *>(w->scale);
  a.bias = static_cast<const uint16_t *>(w->bias);
  a.x = x;
  a.xs = x_scale;
  a.out = out;
  a.xld = x_stride;
  a.old = out_stride;
  a.T = T;
  a.n = w->n;
  a.k = w->k;
  a.xs_cols = cols;
  a.xs_shift = x_group == 0 ? 31 : x_group == 64 ? 0 : 1;
  a.qbf16 = w->qparam_dtype == MOE_BF16;
  a.x_type = int8 ? LinX::Int8 : x_dtype == MOE_BF16 ? LinX::Bf16 : LinX::Fp16;
  a.out_type = out_dtype == MOE_FP32 ? LinOut::Fp32 : out_dtype == MOE_BF16 ? LinOut::Bf16 : LinOut::Fp16;
  return launch_linear(a, stream) == hipSuccess ? MOE_OK : MOE_ERR_HIP;
}

moe_status moe_sample_workspace(int64_t R, int32_t V, size_t *bytes) {
  if (!bytes) return MOE_ERR_NULL;
  if (R < 0 || R > 65535) return MOE_ERR_TOKENS;
  if (V < 1 || V > 1 << 20) return MOE_ERR_SHAPE;
  *bytes = R ? sample_ws(R, V).total : 0;
  return MOE_OK;
}

moe_status moe_sample(int64_t R, int32_t V, const void *logits, int64_t row_stride, moe_dtype dtype, const float *u,
                      const float *temperature, const int32_t *top_k, const float *top_p, const float *min_p,
                      int32_t *token, float *prob, void *workspace, size_t workspace_bytes, hipStream_t stream) {
  if (R < 0 || R > 65535) return MOE_ERR_TOKENS;
  if (V < 1 || V > 1 << 20 || row_stride < 0 || row_stride > int64_t(1) << 38) return MOE_ERR_SHAPE;
  if (dtype != MOE_FP32 && dtype != MOE_BF16 && dtype != MOE_FP16) return MOE_ERR_DTYPE;
  if (R == 0) return MOE_OK;
  if (!logits || !u || !token) return MOE_ERR_NULL;
  const int size = dtype == MOE_FP32 ? 4 : 2;
  if (!aligned(logits, size)) return MOE_ERR_ALIGN;
  for (const void *p : {(const void *)u, (const void *)temperature, (const void *)top_k, (const void *)top_p,
                        (const void *)min_p, (const void *)token, (const void *)prob})
    if (!aligned(p, 4)) return MOE_ERR_ALIGN;
  const SampleWs ws = sample_ws(R, V);
  if (!workspace || workspace_bytes < ws.total) return MOE_ERR_WORKSPACE;
  if (!aligned(workspace, 256)) return MOE_ERR_ALIGN;
  const uint64_t n = 4 * (uint64_t)R;
  const Span st{token, n}, sp{prob, n}, sw{workspace, ws.total};
  const Span read[] = {{logits, (uint64_t)(((R - 1) * row_stride + V) * size)}, {u, n}, {temperature, n}, {top_k, n}, {top_p, n}, {min_p, n}};
  for (const Span &w : {st, sp, sw})
    for (const Span &r : read)
      if (overlap(w, r)) return MOE_ERR_ALIAS;
  if (overlap(st, sp) || overlap(st, sw) || overlap(sp, sw)) return MOE_ERR_ALIAS;
  const moe_status dev = device_ok();
  if (dev != MOE_OK) return dev;
  SampleArgs a{};
  a.logits = logits;
  a.ld = row_stride;
  a.type = dtype == MOE_FP32 ? 0 : dtype == MOE_BF16 ? 1 : 2;
  a.u = u;
  a.temperature = temperature;
  a.top_k = top_k;
  a.top_p = top_p;
  a.min_p = min_p;
  a.token = token;
  a.prob = prob;
  a.R = (int)R;
  a.V = V;
  a.C = ws.chunks;
  int log2v = 0;
  while (1 << log2v < V) ++log2v;
  a.bits = 62 - log2v < 51 ? 62 - log2v : 51;
  char *base = static_cast<char *>(workspace);
  a.chunk = reinterpret_cast<SampleChunk *>(base);
  a.mass = reinterpret_cast<uint64_t *>(base + ws.mass);
  a.count = reinterpret_cast<uint32_t *>(base + ws.count);
  a.row = reinterpret_cast<SampleRow *>(base + ws.row);
  a.kept = reinterpret_cast<uint64_t *>(base + ws.kept);
  a.list = reinterpret_cast<uint64_t *>(base + ws.list);
  a.room = ws.room;
  return launch_sample(a, stream) == hipSuccess ? MOE_OK : MOE_ERR_HIP;
}

}  // extern "C"
