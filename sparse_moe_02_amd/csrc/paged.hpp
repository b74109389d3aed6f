// Device helpers shared by the kernels that read a ragged batch and its paged cache.
#pragma once

#include "common.hpp"
#include "serve.hpp"

namespace moe {

// Largest b in [0, n) with f(b) <= x, for an ascending f with f(0) <= x, by a whole wave: 64
// candidates per step, so 64 sequences take one round of loads and 4096 take two.
template <class F>
__device__ __forceinline__ int wave_find(int n, int64_t x, F f) {
  const int lane = threadIdx.x & 63;
  int lo = 0, len = n;
  while (len > 1) {
    const int step = (len + 63) >> 6;
    const int off = lane * step;
    const bool below = off < len && f(lo + off) <= x;
    // lane 0 counts as below, so the result stays in range whatever f returns
    const int cnt = max(1, (int)__popcll(__ballot(below)));
    lo += (cnt - 1) * step;
    len = min(step, len - (cnt - 1) * step);
  }
  return __builtin_amdgcn_readfirstlane(lo);
}

// Table row of batch sequence b, or -1.
__device__ __forceinline__ int batch_row(const Batch &b, int i) {
  const int r = b.row ? b.row[i] : i;
  return (unsigned)r < (unsigned)b.n_rows ? r : -1;
}

}  // namespace moe
