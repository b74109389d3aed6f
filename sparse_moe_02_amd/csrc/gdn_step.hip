// Gated delta rule, one token each of many sequences ("Optimizing on-device inference for
// Apple Silicon", section "Decode > Reduce intermediate and state traffic").
//
// Per value head, with S the state before the token (rows j = value channels):
//     c_j = beta (v_j - alpha S_j.k),  o_j = alpha S_j.q + c_j (k.q),  S_j <- alpha S_j + c_j k,
// which is S <- alpha S (I - beta k k^T) + beta v k^T, o = S q with both products taken from
// the old state, so a row of S is read once, used, and written once.
//
// Bound: memory (8 bytes per state element and slot, 64 KiB per head each way; 7 flops per
// element).  A 16-lane group holds one state row at a time (8 fp32 per lane) and reduces its
// two dots with DPP; a workgroup of four waves takes 16 x kRowsPer channels of one head, all
// of its state loads in flight at once.
//
// Rows of one slot are applied in row order: the workgroup of the slot's first row takes
// them all, the state staying in registers; the workgroups of the others end.  A decay of 0 takes
// the old state as zeros, whatever it holds (0 times NaN is no zero).
#include "serve.hpp"
#include "common.hpp"
#include "kernels.hpp"

#pragma clang fp contract(off)

namespace moe {

namespace {

constexpr int kD = kGdnDim;
constexpr int kThreads = 256;

__device__ __forceinline__ void unpack8(uint4 w, float *o) {
  o[0] = bf16_lo(w.x); o[1] = bf16_hi(w.x); o[2] = bf16_lo(w.y); o[3] = bf16_hi(w.y);
  o[4] = bf16_lo(w.z); o[5] = bf16_hi(w.z); o[6] = bf16_lo(w.w); o[7] = bf16_hi(w.w);
}

// kRowsPer state rows per 16-lane group: 16 * kRowsPer channels per workgroup.
template <int kRowsPer>
__global__ void __launch_bounds__(kThreads) k_gdn_step(GdnStepArgs a) {
  __shared__ int found;
  constexpr int kParts = kD / (16 * kRowsPer);
  const int tid = threadIdx.x;
  const int part = blockIdx.x % kParts, h = blockIdx.x / kParts % a.hv;
  int r = blockIdx.x / kParts / a.hv;
  const int slot = a.slot[r];
  const int grp = tid >> 4, l = tid & 15;
  const int c0 = part * 16 * kRowsPer;
  if ((unsigned)slot >= (unsigned)a.n_slots) {  // padding: zeros
    if (tid < 16 * kRowsPer) a.out[((int64_t)r * a.hv + h) * kD + c0 + tid] = 0;
    return;
  }
  // the state rows of this group: channels c0 + i * 16 + grp; lane l holds elements
  // 4l..4l+3 and 64+4l..64+4l+3
  float st[kRowsPer][8];
  float *sp = a.state + (((int64_t)slot * a.hv + h) * kD + c0 + grp) * kD + 4 * l;
#pragma unroll
  for (int i = 0; i < kRowsPer; ++i) {
    *(float4 *)&st[i][0] = *(const float4 *)(sp + i * 16 * kD);
    *(float4 *)&st[i][4] = *(const float4 *)(sp + i * 16 * kD + 64);
  }
  int earlier = 0;
  for (int i = tid; i < r; i += kThreads) earlier |= a.slot[i] == slot;
  if (__syncthreads_or(earlier)) return;  // an earlier row's workgroup has this one

  const int kh = h / (a.hv / a.hk);
  while (true) {
    const uint16_t *kp = a.k + ((int64_t)r * a.hk + kh) * kD + 4 * l;
    const uint16_t *qp = a.q + ((int64_t)r * a.hk + kh) * kD + 4 * l;
    const uint2 k0 = *(const uint2 *)kp, k1 = *(const uint2 *)(kp + 64);
    const uint2 q0 = *(const uint2 *)qp, q1 = *(const uint2 *)(qp + 64);
    float kf[8], qf[8];
    unpack8(make_uint4(k0.x, k0.y, k1.x, k1.y), kf);
    unpack8(make_uint4(q0.x, q0.y, q1.x, q1.y), qf);
    const float alpha = a.alpha[(int64_t)r * a.hv + h], beta = a.beta[(int64_t)r * a.hv + h];
    if (alpha == 0.0f) {
#pragma unroll
      for (int i = 0; i < kRowsPer; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e) st[i][e] = 0.0f;
    }
    const int64_t ob = ((int64_t)r * a.hv + h) * kD + c0 + grp;
    float kq = 0.0f;
#pragma unroll
    for (int e = 0; e < 8; ++e) kq = __builtin_fmaf(kf[e], qf[e], kq);
    kq = row16_sum(kq);
#pragma unroll
    for (int i = 0; i < kRowsPer; ++i) {
      float sk0 = 0.0f, sk1 = 0.0f, sq0 = 0.0f, sq1 = 0.0f;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        sk0 = __builtin_fmaf(st[i][e], kf[e], sk0);
        sq0 = __builtin_fmaf(st[i][e], qf[e], sq0);
        sk1 = __builtin_fmaf(st[i][4 + e], kf[4 + e], sk1);
        sq1 = __builtin_fmaf(st[i][4 + e], qf[4 + e], sq1);
      }
      const float sk = row16_sum(sk0 + sk1), sq = row16_sum(sq0 + sq1);
      const float c = beta * __builtin_fmaf(-alpha, sk, bf16_to_f32(a.v[ob + i * 16]));
      if (l == 0) a.out[ob + i * 16] = f32_to_bf16(__builtin_fmaf(alpha, sq, c * kq));
#pragma unroll
      for (int e = 0; e < 8; ++e) st[i][e] = __builtin_fmaf(c, kf[e], alpha * st[i][e]);
    }
    // the slot's next row
    int next = a.R;
    for (int i = r + 1 + tid; i < a.R; i += kThreads)
      if (a.slot[i] == slot) {
        next = i;
        break;
      }
    if (!__syncthreads_or(next < a.R)) break;
    if (tid == 0) found = a.R;
    __syncthreads();
    if (next < a.R) atomicMin(&found, next);
    __syncthreads();
    r = found;
    __syncthreads();
  }
#pragma unroll
  for (int i = 0; i < kRowsPer; ++i) {
    *(float4 *)(sp + i * 16 * kD) = *(const float4 *)&st[i][0];
    *(float4 *)(sp + i * 16 * kD + 64) = *(const float4 *)&st[i][4];
  }
}

}  // namespace

hipError_t launch_gdn_step(const GdnStepArgs &a, hipStream_t s) {
  if (a.R <= 0) return hipSuccess;
  hipLaunchKernelGGL(k_gdn_step<4>, dim3(a.R * a.hv * 2), dim3(kThreads), 0, s, a);
  return hipGetLastError();
}

}  // namespace moe
