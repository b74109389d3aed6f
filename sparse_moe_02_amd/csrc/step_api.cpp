// Host side of the C ABI declared in include/norm.h: argument checks and launches.  Every check
// precedes every launch.
#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdint>

#include "../../include/norm.h"
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

}  // extern "C"
