// Bookkeeping of the paged cache: grow, fork, free, compact, copy.
//
// A call is a plan over the requests (checks, fresh pages needed and their prefix sums), a
// count of free pages by groups of kPageGroup, and an application in which every workgroup
// takes its own share: the page of rank r among the free ones goes to the request whose prefix
// sums bracket r.  A group's workgroup knows the rank of its first free page from the counts before
// it; where requests look for their pages instead (fork), a group lists its first ones.  Ranks
// are positions, not arrival order: results are the same on every run, and refs of shared pages
// change by integer atomics, whose order does not matter.
//
// Bound: latency for the tables (two launches of small integer work: 256 sequences growing in a
// pool of 65536 pages take 9.2 us); memory for the pages copied (16 bytes per lane, kCopyVecs in
// flight): a compaction that moves some 450 pages of 32 KB in 20 planes takes 121 us for them,
// 4.9 TB/s, and 32 forks that copy a page each in as many planes 14.4 us for everything.
#include "paged.hpp"

namespace moe {

namespace {

constexpr int kThreads = 256;
constexpr int kPlanThreads = 1024;
constexpr int kNear = 2048;  // requests whose prefix sums are searched in LDS
constexpr int kCopyVecs = 4;                                  // 16-byte vectors a lane has in flight
constexpr int64_t kCopyChunk = int64_t(kThreads) * 16 * kCopyVecs;  // bytes per workgroup step

enum Status { kOk = 0, kShape = 2, kAlloc = 10 };  // moe_status

__device__ __forceinline__ int pages_of(int len, int shift) {
  return (int)(((int64_t)len + (1 << shift) - 1) >> shift);
}

// Sum over a workgroup; every thread gets it.  `s`: one int per wave.
template <int N>
__device__ __forceinline__ int block_sum(int v, int *s) {
  const int tid = threadIdx.x;
  v = __builtin_amdgcn_readlane(wave_incl_scan(v), 63);
  if ((tid & 63) == 0) s[tid >> 6] = v;
  __syncthreads();
  int t = 0;
#pragma unroll
  for (int i = 0; i < N / 64; ++i) t += s[i];
  __syncthreads();
  return t;
}
// Exclusive prefix sum over a workgroup; total gets the sum.
template <int N>
__device__ __forceinline__ int block_excl(int v, int *s, int &total) {
  const int tid = threadIdx.x, w = tid >> 6;
  const int inc = wave_incl_scan(v);
  if ((tid & 63) == 63) s[w] = inc;
  __syncthreads();
  int before = 0;
  total = 0;
#pragma unroll
  for (int i = 0; i < N / 64; ++i) {
    if (i < w) before += s[i];
    total += s[i];
  }
  __syncthreads();
  return before + inc - v;
}

// Whether sequence s of the input pool has a length its table row can hold.
__device__ __forceinline__ bool len_ok(const PageArgs &a, int64_t len) {
  return len >= 0 && len <= (int64_t)a.cols << a.page_shift;
}

// The requests: checks and the fresh pages each needs.
template <PageOp OP>
__device__ void plan(const PageArgs &a) {
  __shared__ uint32_t seen[65536 / 32];
  __shared__ int sums[kPlanThreads / 64];
  const int tid = threadIdx.x;
  for (int i = tid; i < 65536 / 32; i += kPlanThreads) seen[i] = 0;
  __syncthreads();
  bool wrong = false;
  int at = 0;  // fresh pages needed so far
  for (int i0 = 0; i0 < a.n; i0 += kPlanThreads) {
    const int i = i0 + tid;
    int need = 0, col = 0, longer = 0;
    if (i < a.n) {
      const int s = a.a[i];
      const int d = OP == PageOp::Fork ? a.b[i] : s;  // the sequence that changes
      if ((unsigned)s >= (unsigned)a.n_seqs || (unsigned)d >= (unsigned)a.n_seqs) {
        wrong = true;
      } else {
        wrong |= (atomicOr(&seen[d >> 5], 1u << (d & 31)) >> (d & 31)) & 1;
        const int len = a.in.len[s];
        wrong |= !len_ok(a, len);
        if (OP == PageOp::Grow) {
          const int more = a.b[i];
          if (!len_ok(a, len) || more < 0 || !len_ok(a, (int64_t)len + more)) {
            wrong = true;
          } else {
            longer = len + more;
            col = pages_of(len, a.page_shift);
            need = pages_of(longer, a.page_shift) - col;
          }
        } else if (OP == PageOp::Fork) {
          wrong |= a.in.len[d] != 0;
          need = (len & ((1 << a.page_shift) - 1)) != 0;
        }
      }
    }
    if (OP != PageOp::Free) {
      int total;
      const int before = block_excl<kPlanThreads>(need, sums, total);
      if (i < a.n) {
        a.base[i] = at + before;
        if (OP == PageOp::Grow) {
          a.col[i] = col;
          a.longer[i] = longer;
        }
      }
      at += total;
    }
  }
  if (OP == PageOp::Fork) {  // no source among the destinations
    __syncthreads();
    for (int i = tid; i < a.n; i += kPlanThreads) {
      const int s = a.a[i];
      if ((unsigned)s < (unsigned)a.n_seqs) wrong |= (seen[s >> 5] >> (s & 31)) & 1;
    }
  }
  const int any = __syncthreads_or(wrong);
  if (tid == 0) {
    a.hdr[0] = any ? kShape : kOk;
    a.hdr[1] = at;
    if (OP != PageOp::Free && OP != PageOp::Compact) a.base[a.n] = at;
  }
}

// First launch.  Workgroup 0 plans; then one workgroup per group counts free pages and copies
// the group's refs; then one per row copies the row; then one per request (per row where
// compacting) checks the table entries that the call will use.
template <PageOp OP>
__global__ void __launch_bounds__(kPlanThreads) k_pages_plan(PageArgs a) {
  __shared__ int sums[kPlanThreads / 64];
  const int tid = threadIdx.x;
  const int groups = (a.n_pages + kPageGroup - 1) / kPageGroup;
  const bool copy = a.out.table != a.in.table;
  int w = blockIdx.x;
  if (w == 0) {
    if (OP == PageOp::Compact) {
      if (tid == 0) a.hdr[0] = kOk;
    } else {
      plan<OP>(a);
    }
    return;
  }
  w -= 1;
  if (w < groups) {
    constexpr int kSteps = kPageGroup / kPlanThreads;
    const int p0 = w * kPageGroup + tid;
    int refs[kSteps], n = 0;
#pragma unroll
    for (int q = 0; q < kSteps; ++q) {
      const int p = p0 + q * kPlanThreads;
      refs[q] = p < a.n_pages ? a.in.refs[p] : 1;
      n += refs[q] <= 0;
      if (copy && p < a.n_pages) a.out.refs[p] = refs[q];
    }
    if (OP == PageOp::Fork) {  // the group's free pages, in order
      n = 0;
#pragma unroll
      for (int q = 0; q < kSteps; ++q) {
        int total;
        const int r = n + block_excl<kPlanThreads>(refs[q] <= 0, sums, total);
        if (refs[q] <= 0 && r < a.n) a.fresh[w * kPageGroup + r] = p0 + q * kPlanThreads;
        n += total;
      }
    } else {
      n = block_sum<kPlanThreads>(n, sums);
    }
    if (tid == 0) a.free_n[w] = n;
    return;
  }
  w -= groups;
  if (copy) {
    if (w < a.n_seqs) {
      const int64_t o = (int64_t)w * a.cols;
      for (int c = tid; c < a.cols; c += kPlanThreads) a.out.table[o + c] = a.in.table[o + c];
      if (tid == 0) a.out.len[w] = a.in.len[w];
      return;
    }
    w -= a.n_seqs;
  }
  if (OP == PageOp::Grow) return;
  const int s = OP == PageOp::Compact ? w : a.a[w];
  bool bad = true;
  if ((unsigned)s < (unsigned)a.n_seqs && len_ok(a, a.in.len[s])) {
    bad = false;
    const int n = pages_of(a.in.len[s], a.page_shift);
    for (int c = tid; c < n; c += kPlanThreads)
      bad |= (unsigned)a.in.table[(int64_t)s * a.cols + c] >= (unsigned)a.n_pages;
  }
  const int any = __syncthreads_or(bad);
  if (tid == 0) a.bad[w] = any;
}

// Free pages before group w, and in the pool.
__device__ __forceinline__ int free_before(const PageArgs &a, int w, int groups, int *sums, int &total) {
  int before = 0, all = 0;
  for (int i = threadIdx.x; i < groups; i += kThreads) {
    const int n = a.free_n[i];
    all += n;
    before += i < w ? n : 0;
  }
  total = block_sum<kThreads>(all, sums);
  return block_sum<kThreads>(before, sums);
}

// The call's status, the same in every workgroup.
template <PageOp OP>
__device__ __forceinline__ int status(const PageArgs &a, int total_free) {
  bool bad = false;
  if (OP != PageOp::Grow)
    for (int i = threadIdx.x; i < (OP == PageOp::Compact ? a.n_seqs : a.n); i += kThreads) bad |= a.bad[i] != 0;
  if (__syncthreads_or(bad) || a.hdr[0] != kOk) return kShape;
  if ((OP == PageOp::Grow || OP == PageOp::Fork) && a.hdr[1] > total_free) return kAlloc;
  return kOk;
}

// Second launch (Fork has its own).  One workgroup per group hands out its free pages (compact:
// lists its free pages and its pages that move); then one per request applies it.
template <PageOp OP>
__global__ void __launch_bounds__(kThreads) k_pages_apply(PageArgs a) {
  __shared__ int sums[kThreads / 64];
  __shared__ int counts[64];
  __shared__ int near_base[OP == PageOp::Compact ? 1 : kNear];
  const int tid = threadIdx.x;
  const int groups = (a.n_pages + kPageGroup - 1) / kPageGroup;
  const int w = blockIdx.x;
  // the group's pages, kThreads at a time: which are free (read before anything is known of the
  // call, like the prefix sums of the requests, for the searches below)
  constexpr int kSteps = kPageGroup / kThreads, kW = kThreads / 64;
  static_assert(kSteps * kW == 64, "a wave scans the counts");
  const int p0 = w * kPageGroup, lane = tid & 63;
  const bool near = a.n < kNear;
  uint32_t free_bits = 0, in_bits = 0;
  if (OP != PageOp::Free && w < groups) {
#pragma unroll
    for (int q = 0; q < kSteps; ++q) {
      const int p = p0 + q * kThreads + tid;
      const int refs = a.in.refs[min(p, a.n_pages - 1)];
      if (p < a.n_pages) in_bits |= 1u << q;
      if (p < a.n_pages && refs <= 0) free_bits |= 1u << q;
    }
    if (OP != PageOp::Compact && near)
      for (int i = tid; i < a.n; i += kThreads) near_base[i] = a.base[i];
  }
  int total;
  const int rank = free_before(a, w, groups, sums, total);
  const int st = status<OP>(a, total);
  if (w == 0 && tid == 0) {
    if (OP == PageOp::Compact) a.hdr[1] = a.n_pages - total;
    // the group of page `used` writes the number of pages that move, if there are free pages
    if (OP == PageOp::Compact && (st != kOk || total == 0)) a.hdr[2] = 0;
    if (st != kOk) atomicCAS(a.error, 0, st);
  }
  if (st != kOk) return;
  if (OP == PageOp::Grow && w == 0)
    for (int i = tid; i < a.n; i += kThreads) a.out.len[a.a[i]] = a.longer[i];
  if (w < groups) {
    if (OP == PageOp::Free) return;
    const int used = a.n_pages - total;  // compact: pages below this number stay
    const int need = OP == PageOp::Compact ? 0 : a.hdr[1];
    if (OP != PageOp::Compact && rank >= need) return;
#pragma unroll
    for (int q = 0; q < kSteps; ++q) {
      const int n = __popcll(__ballot(free_bits >> q & 1));
      if (lane == 0) counts[q * kW + (tid >> 6)] = n;
    }
    __syncthreads();
    const int mine = counts[lane], before = wave_incl_scan(mine) - mine;  // of (step, wave) = lane
    for (int q = 0; q < kSteps; ++q) {
      const bool is_free = free_bits >> q & 1;
      const uint64_t ahead = __ballot(is_free) & ((uint64_t(1) << lane) - 1);
      const int r = rank + __shfl(before, q * kW + (tid >> 6), 64) + (int)__popcll(ahead);
      if (!(in_bits >> q & 1)) continue;
      const int p = p0 + q * kThreads + tid;
      if (OP == PageOp::Compact) {
        // free pages below `used` take, rank by rank, the used ones at and behind it
        if (p == used) a.hdr[2] = r;
        if (is_free && p < used) a.fresh[r] = p;
        // ranked from the pool's end, where no other group's count is missing
        if (!is_free && p >= used) a.moved[a.n_pages - 1 - p - (total - r)] = p;
      } else if (is_free && r < need) {
        // the request whose range of ranks holds r: the last one with base <= r
        int lo = 0, len = a.n;
        while (len > 1) {
          const int half = len / 2;
          if ((near ? near_base[lo + half] : a.base[lo + half]) <= r) {
            lo += half;
            len -= half;
          } else {
            len = half;
          }
        }
        a.out.table[(int64_t)a.a[lo] * a.cols + a.col[lo] + (r - a.base[lo])] = p;
        a.out.refs[p] = 1;
      }
    }
    return;
  }
  if (OP == PageOp::Free) {
    const int s = a.a[w - groups], n = pages_of(a.in.len[s], a.page_shift);
    for (int c = tid; c < n; c += kThreads) atomicAdd(&a.out.refs[a.in.table[(int64_t)s * a.cols + c]], -1);
    __syncthreads();  // nobody else reads this length: sequences end once
    if (tid == 0) a.out.len[s] = 0;
  }
}

// Copy `bytes` of one page, the part that starts at `at`.
__device__ __forceinline__ void copy_part(const PageMem &m, int plane, int src, int dst, int64_t at) {
  const int64_t o = plane * m.plane + at + threadIdx.x * 16;
  const uint8_t *s = m.base + o + src * m.page;
  uint8_t *d = m.base + o + dst * m.page;
  u32x4 v[kCopyVecs];
#pragma unroll
  for (int i = 0; i < kCopyVecs; ++i)
    if (at + threadIdx.x * 16 + i * kThreads * 16 < m.bytes) v[i] = *(const u32x4 *)(s + i * kThreads * 16);
#pragma unroll
  for (int i = 0; i < kCopyVecs; ++i)
    if (at + threadIdx.x * 16 + i * kThreads * 16 < m.bytes) *(u32x4 *)(d + i * kThreads * 16) = v[i];
}

// Walks this workgroup's share of `pairs` copies in every plane; the first `others` workgroups
// do something else.
template <class F>
__device__ __forceinline__ void copy_pages(const PageMem &m, int64_t pairs, int others, F pair) {
  const int64_t parts = (m.bytes + kCopyChunk - 1) / kCopyChunk, per = parts * m.n_planes;
  for (int64_t x = blockIdx.x - others; x < pairs * per; x += gridDim.x - others) {
    const int64_t i = x / per, y = x % per;
    int src, dst;
    if (pair(i, src, dst)) copy_part(m, (int)(y / parts), src, dst, y % parts * kCopyChunk);
  }
}

// The free page of a rank, by a whole wave, from the lists of the groups.
__device__ __forceinline__ int fresh_page(const PageArgs &a, int rank, int groups) {
  const int lane = threadIdx.x & 63;
  for (int g = 0;; g += 64) {
    const int n = g + lane < groups ? a.free_n[g + lane] : 0, upto = wave_incl_scan(n);
    const uint64_t behind = __ballot(upto > rank);
    if (behind || g + 64 >= groups) {
      const int l = behind ? __builtin_ctzll(behind) : 0;
      return a.fresh[(int64_t)(g + l) * kPageGroup + rank - __builtin_amdgcn_readlane(upto - n, l)];
    }
    rank -= __builtin_amdgcn_readlane(upto, 63);
  }
}

// Fork's second launch: one workgroup per request shares its full pages, the others copy last
// pages that are not full.  Both find a fresh page in the lists of the first launch, so the copies
// need not wait for a launch of their own (32 forks, 17.5 -> 14.4 us).
__global__ void __launch_bounds__(kThreads) k_pages_fork(PageArgs a) {
  __shared__ int sums[kThreads / 64];
  const int tid = threadIdx.x;
  const int groups = (a.n_pages + kPageGroup - 1) / kPageGroup;
  int total;
  free_before(a, 0, groups, sums, total);
  const int st = status<PageOp::Fork>(a, total);
  if (blockIdx.x == 0 && tid == 0 && st != kOk) atomicCAS(a.error, 0, st);
  if (st != kOk) return;
  const int i = blockIdx.x;
  if (i >= a.n) {
    copy_pages(a.mem, a.n, a.n, [&](int64_t i, int &src, int &dst) {
      if (a.base[i + 1] == a.base[i]) return false;
      const int s = a.a[i];
      src = a.in.table[(int64_t)s * a.cols + (a.in.len[s] >> a.page_shift)];
      dst = fresh_page(a, a.base[i], groups);
      return true;
    });
    return;
  }
  const int s = a.a[i], len = a.in.len[s], n = len >> a.page_shift;
  const int64_t to = (int64_t)a.b[i] * a.cols;
  for (int c = tid; c < n; c += kThreads) {
    const int p = a.in.table[(int64_t)s * a.cols + c];
    atomicAdd(&a.out.refs[p], 1);
    a.out.table[to + c] = p;
  }
  if (a.base[i + 1] != a.base[i]) {
    const int p = fresh_page(a, a.base[i], groups);
    if (tid == 0) {
      a.out.table[to + n] = p;
      a.out.refs[p] = 1;
    }
  }
  if (tid == 0) a.out.len[a.b[i]] = len;  // (nobody reads it: a destination is no source)
}

// Compact: pages, refs and tables follow the lists.
__global__ void __launch_bounds__(kThreads) k_pages_move(PageArgs a) {
  const int n = a.hdr[2], used = a.hdr[1];
  if (n == 0) return;
  for (int64_t i = blockIdx.x * (int64_t)kThreads + threadIdx.x; i < n; i += (int64_t)gridDim.x * kThreads) {
    const int from = a.moved[n - 1 - i];
    a.out.refs[a.fresh[i]] = a.in.refs[from];
    a.out.refs[from] = 0;
  }
  for (int64_t s = blockIdx.x; s < a.n_seqs; s += gridDim.x) {
    const int pages = pages_of(a.in.len[s], a.page_shift);
    for (int c = threadIdx.x; c < pages; c += kThreads) {
      const int p = a.in.table[s * a.cols + c];
      if (p < used) continue;
      int lo = 0, len = n;  // by rank, moved pages ascend
      while (len > 1) {
        const int half = len / 2;
        if (a.moved[n - 1 - lo - half] <= p) {
          lo += half;
          len -= half;
        } else {
          len = half;
        }
      }
      if (a.moved[n - 1 - lo] == p) a.out.table[s * a.cols + c] = a.fresh[lo];
    }
  }
  copy_pages(a.mem, n, 0, [&](int64_t i, int &src, int &dst) {
    src = a.moved[n - 1 - i];
    dst = a.fresh[i];
    return true;
  });
}

__global__ void __launch_bounds__(kThreads) k_pages_copy(PageMem m, int n_pages, int n, const int32_t *from, const int32_t *to) {
  copy_pages(m, n, 0, [&](int64_t i, int &src, int &dst) {
    src = from[i];
    dst = to[i];
    return (unsigned)src < (unsigned)n_pages && (unsigned)dst < (unsigned)n_pages;
  });
}

constexpr int kCopyGrid = 2048;

int copy_grid(const PageMem &m, int64_t pairs) {
  const int64_t parts = (m.bytes + kCopyChunk - 1) / kCopyChunk * m.n_planes;
  return (int)(pairs * parts < kCopyGrid ? pairs * parts : kCopyGrid);
}

template <PageOp OP>
hipError_t launch(const PageArgs &a, hipStream_t s) {
  const int groups = (a.n_pages + kPageGroup - 1) / kPageGroup;
  const int rows = a.out.table != a.in.table ? a.n_seqs : 0;
  const int checks = OP == PageOp::Compact ? a.n_seqs : OP == PageOp::Grow ? 0 : a.n;
  hipLaunchKernelGGL(k_pages_plan<OP>, dim3(1 + groups + rows + checks), dim3(kPlanThreads), 0, s, a);
  if (OP == PageOp::Fork) {
    if (a.n > 0) hipLaunchKernelGGL(k_pages_fork, dim3(a.n + copy_grid(a.mem, a.n)), dim3(kThreads), 0, s, a);
    return hipGetLastError();
  }
  hipLaunchKernelGGL(k_pages_apply<OP>, dim3(groups + (OP == PageOp::Free ? a.n : 0)), dim3(kThreads), 0, s, a);
  if (OP == PageOp::Compact)
    hipLaunchKernelGGL(k_pages_move, dim3(copy_grid(a.mem, a.n_pages)), dim3(kThreads), 0, s, a);
  return hipGetLastError();
}

}  // namespace

PageWs page_ws(int n_seqs, int n_pages, int n) {
  PageWs w{};
  size_t o = 256;
  auto take = [&](size_t ints) {
    const size_t at = o;
    o = (o + 4 * ints + 255) & ~(size_t)255;
    return at;
  };
  w.free_n = take((n_pages + kPageGroup - 1) / kPageGroup);
  w.bad = take(n > n_seqs ? n : n_seqs);
  w.base = take((size_t)n + 1);
  w.col = take(n);
  w.longer = take(n);
  w.fresh = take(n_pages);
  w.moved = take(n_pages);
  w.total = o;
  return w;
}

hipError_t launch_pages(PageOp op, const PageArgs &a, hipStream_t s) {
  switch (op) {
    case PageOp::Grow: return launch<PageOp::Grow>(a, s);
    case PageOp::Fork: return launch<PageOp::Fork>(a, s);
    case PageOp::Free: return launch<PageOp::Free>(a, s);
    case PageOp::Compact: return launch<PageOp::Compact>(a, s);
  }
  return hipErrorInvalidValue;
}

hipError_t launch_pages_copy(const PageMem &m, int n_pages, int n, const int32_t *src, const int32_t *dst, hipStream_t s) {
  if (n <= 0) return hipSuccess;
  hipLaunchKernelGGL(k_pages_copy, dim3(copy_grid(m, n)), dim3(kThreads), 0, s, m, n_pages, n, src, dst);
  return hipGetLastError();
}

}  // namespace moe
