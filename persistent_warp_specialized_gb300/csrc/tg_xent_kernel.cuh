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

// One warp a row.  Lanes take every 32nd slot; the largest maximum first, then the scaled sums in a
// fixed order.
__global__ void __launch_bounds__(256) xent_join_kernel(const XentJoinParams p) {
  grid_dependency_wait();
  grid_launch_dependents();
  const uint32_t lane = threadIdx.x & 31u;
  const uint64_t row = (static_cast<uint64_t>(blockIdx.x) * blockDim.x + threadIdx.x) / 32u;
  if (row >= p.rows) return;
  const float2* src = p.stats + row * p.slots;
  float top = -INFINITY;
  for (uint32_t i = lane; i < p.slots; i += 32u) top = fmaxf(top, src[i].x);
#pragma unroll
  for (uint32_t o = 16; o > 0; o /= 2) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  const float base = top == -INFINITY ? 0.0f : top;
  float sum = 0.0f;
  for (uint32_t i = lane; i < p.slots; i += 32u) {
    const float2 c = src[i];
    sum += c.y * expf(c.x - base);
  }
#pragma unroll
  for (uint32_t o = 16; o > 0; o /= 2) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if (lane == 0) {
    const float lse = top + logf(sum);
    const TargetKind kind = target_kind(p.targets[row], p.ignore, p.vocab);
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
