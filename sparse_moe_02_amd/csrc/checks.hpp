// Argument checks that the host sides of the serving operators share.
#pragma once

#include <hip/hip_runtime.h>

#include <algorithm>
#include <atomic>
#include <cstdint>
#include <cstring>

#include "../../include/attn.h"
#include "serve.hpp"

namespace moe {

constexpr int64_t kMaxTokens = int64_t(1) << 20;

inline bool aligned(const void *p, uintptr_t n) { return ((uintptr_t)p & (n - 1)) == 0; }

// gfx950 check of the current device, cached per device.
constexpr int kMaxDevs = 64;
inline std::atomic<int> g_dev_ok[kMaxDevs];  // 0 unknown, 1 gfx950, 2 other
inline moe_status device_ok() {
  int dev = 0;
  if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= kMaxDevs) return MOE_ERR_DEVICE;
  int ok = g_dev_ok[dev].load(std::memory_order_relaxed);
  if (ok == 0) {
    hipDeviceProp_t prop;
    if (hipGetDeviceProperties(&prop, dev) != hipSuccess) return MOE_ERR_DEVICE;
    ok = std::strncmp(prop.gcnArchName, "gfx950", 6) == 0 ? 1 : 2;
    g_dev_ok[dev].store(ok, std::memory_order_relaxed);
  }
  return ok == 1 ? MOE_OK : MOE_ERR_DEVICE;
}

// A range of bytes.  Empty ranges overlap nothing.
struct Span {
  const void *p;
  uint64_t n;
};
inline bool overlap(const Span &a, const Span &b) {
  if (!a.p || !b.p || !a.n || !b.n) return false;
  const uintptr_t x = (uintptr_t)a.p, y = (uintptr_t)b.p;
  return x < y + b.n && y < x + a.n;
}

// Dimensions with more than one element, over an innermost one of `inner` elements: no two
// elements share a place where each stride covers the dimensions inside it.
struct Dim {
  int64_t stride, count;
};
inline bool distinct(Dim *d, int n, int64_t inner) {
  std::sort(d, d + n, [](const Dim &a, const Dim &b) { return a.stride < b.stride; });
  __int128 need = inner;
  for (int i = 0; i < n; ++i) {
    if (d[i].count <= 1) continue;
    if (d[i].stride < need) return false;
    need = (__int128)d[i].stride * d[i].count;
    if (need > (__int128)1 << 60) return false;
  }
  return true;
}

// Bytes from p that [T][heads][dim] spans.
inline Span span(const moe_heads &x, int64_t T, int64_t heads, int64_t dim) {
  if (T <= 0 || heads <= 0) return Span{x.p, 0};
  return Span{x.p, (uint64_t)(2 * ((T - 1) * x.token_stride + (heads - 1) * x.head_stride + dim))};
}

// Whether two [T][.][dim] arrays may share elements.  Arrays of one token stride that
// interleave (slices of one projection's rows) are compared within a row.
inline bool heads_overlap(const moe_heads &a, int64_t ha, const moe_heads &b, int64_t hb, int64_t T, int64_t dim) {
  const Span sa = span(a, T, ha, dim), sb = span(b, T, hb, dim);
  if (!overlap(sa, sb)) return false;
  if (a.token_stride != b.token_stride || a.token_stride == 0) return true;
  const int64_t ts = 2 * a.token_stride;
  const int64_t wa = 2 * ((ha - 1) * a.head_stride + dim), wb = 2 * ((hb - 1) * b.head_stride + dim);
  if (wa > ts || wb > ts) return true;
  int64_t d = ((int64_t)((uintptr_t)a.p - (uintptr_t)b.p)) % ts;  // a's row starts d behind one of b's
  if (d < 0) d += ts;
  return !(d >= wb && d + wa <= ts);
}

inline moe_status check_heads(const moe_heads *x) {
  if (!x || !x->p) return MOE_ERR_NULL;
  if (!aligned(x->p, 16)) return MOE_ERR_ALIGN;
  if (x->token_stride < 0 || x->head_stride < 0 || x->token_stride > int64_t(1) << 38 ||
      x->head_stride > int64_t(1) << 38)
    return MOE_ERR_SHAPE;
  if (x->token_stride % 8 || x->head_stride % 8) return MOE_ERR_ALIGN;
  return MOE_OK;
}
inline bool heads_distinct(const moe_heads &x, int64_t T, int64_t heads, int64_t dim) {
  Dim d[2] = {{x.token_stride, T}, {x.head_stride, heads}};
  return distinct(d, 2, dim);
}

inline Heads dev_heads(const moe_heads &x) {
  return Heads{static_cast<uint16_t *>(const_cast<void *>(x.p)), x.token_stride, x.head_stride};
}

}  // namespace moe
