// tg_xent_kernel.cuh -- what the cross entropy does outside the tensor core.
//
// The product's epilogue leaves, for each row and 128 logits, their maximum m and s = sum exp(l - m),
// and the target's logit t.  With M the largest m:  lse = M + log sum s exp(m - M),  loss = lse - t.
#pragma once

#include "tg_linear_kernel.cuh"

namespace tg {

// A row counts where its target is not ``ignore``; a target outside the vocabulary makes NaN of it.
enum TargetKind { kTargetIgnored, kTargetValid, kTargetWrong };
__device__ __forceinline__ TargetKind target_kind(int64_t t, int64_t ignore, uint32_t vocab) {
  if (t == ignore) return kTargetIgnored;
  return t >= 0 && t < static_cast<int64_t>(vocab) ? kTargetValid : kTargetWrong;
}

struct XentJoinParams {
  const float2* stats;
  const float* hit;
  const int64_t* targets;
  int64_t ignore;
  float *loss, *lse;
  uint32_t rows, slots, vocab;
};

// One warp a row.  A lane takes every 32nd slot, four at a time, and keeps a running maximum and the sum
// relative to it; lanes are joined in a fixed order.
__global__ void __launch_bounds__(128) xent_join_kernel(const XentJoinParams p) {
  grid_dependency_wait();
  grid_launch_dependents();
  const uint32_t lane = threadIdx.x & 31u;
  const uint64_t row = (static_cast<uint64_t>(blockIdx.x) * blockDim.x + threadIdx.x) / 32u;
  if (row >= p.rows) return;
  const float2* src = p.stats + row * p.slots;
  const int64_t target = p.targets[row];
  float top = -INFINITY, sum = 0.0f;
  // to a new maximum; where there is none yet the exponentials are 0
  auto join = [](float& top, float& sum, float m, float s) {
    const float t = fmaxf(top, m), base = t == -INFINITY ? 0.0f : t;
    sum = sum * __expf(top - base) + s * __expf(m - base);
    top = t;
  };
  for (uint32_t i = lane; i < p.slots; i += 128u) {
    float2 c[4];
#pragma unroll
    for (uint32_t j = 0; j < 4; ++j)
      c[j] = i + 32u * j < p.slots ? src[i + 32u * j] : make_float2(-INFINITY, 0.0f);
#pragma unroll
    for (uint32_t j = 0; j < 4; ++j) join(top, sum, c[j].x, c[j].y);
  }
#pragma unroll
  for (uint32_t o = 16; o > 0; o /= 2) {
    const float m = __shfl_xor_sync(0xffffffffu, top, o), s = __shfl_xor_sync(0xffffffffu, sum, o);
    join(top, sum, m, s);
  }
  if (lane == 0) {
    const float lse = top + logf(sum);
    const TargetKind kind = target_kind(target, p.ignore, p.vocab);
    p.lse[row] = lse;
    p.loss[row] = kind == kTargetIgnored ? 0.0f
                  : kind == kTargetValid ? lse - p.hit[row]
                                         : __int_as_float(0x7fffffff);
  }
}

struct XentWeightParams {
  const float* dloss;
  const int64_t* targets;
  int64_t ignore;
  float *weight, *alpha;
  uint32_t rows, vocab;
  float whole;             // the largest weight
};

// weight = whole dloss / d for rows that count, with d the largest |dloss| among them; 0 for ignored ones,
// NaN for wrong targets; alpha = d / whole.  Gradients of logits are rounded relative to d: where dloss is
// the same in every row, a target's -1 is exact instead of off by one rounding in all rows alike (4096 rows
// of 65536 words, bf16: dx 2.9e-3 off, now 1.9e-3; its own rounding makes 1.7e-3).  whole: 1 in bf16; in fp16, which has few exponents,
// 2^15, so that probabilities 2^29 times smaller keep all their bits.  One block: rows are few beside the
// products that follow.
__global__ void __launch_bounds__(1024) xent_weight_kernel(const XentWeightParams p) {
  __shared__ float part[32];
  grid_dependency_wait();
  grid_launch_dependents();
  float top = 0.0f;
  for (uint32_t r = threadIdx.x; r < p.rows; r += blockDim.x)
    if (target_kind(p.targets[r], p.ignore, p.vocab) == kTargetValid)
      top = fmaxf(top, fabsf(p.dloss[r]));
#pragma unroll
  for (uint32_t o = 16; o > 0; o /= 2) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  if ((threadIdx.x & 31u) == 0) part[threadIdx.x / 32u] = top;
  __syncthreads();
  top = part[threadIdx.x & 31u];
#pragma unroll
  for (uint32_t o = 16; o > 0; o /= 2) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  // nothing to be relative to: no gradient at all, or an infinite one
  const bool plain = !(top > 0.0f && top < INFINITY);
  if (threadIdx.x == 0) *p.alpha = plain ? 1.0f : top / p.whole;
  for (uint32_t r = threadIdx.x; r < p.rows; r += blockDim.x) {
    const TargetKind kind = target_kind(p.targets[r], p.ignore, p.vocab);
    const float d = kind == kTargetValid ? p.dloss[r] : 0.0f;
    p.weight[r] = kind == kTargetWrong ? __int_as_float(0x7fffffff)
                  : plain              ? d
                                       : d / top * p.whole;
  }
}

}  // namespace tg
