// tg_xent_kernel.cuh -- what the cross entropy does outside the tensor core.
//
// The product's epilogue leaves, for each row and 128 logits, their maximum m and s = sum exp(l - m),
// and the target's logit t.  With M the largest m:  lse = M + log sum s exp(m - M),  loss = lse - t.
#pragma once

#include "tg_linear_kernel.cuh"

namespace tg {

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

}  // namespace tg
