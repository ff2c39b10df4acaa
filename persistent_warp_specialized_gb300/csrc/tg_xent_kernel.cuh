// tg_xent_kernel.cuh -- what the cross entropy does outside the tensor core.
//
// The product's epilogue leaves, for each row and 64 (few rows: 128) logits, their maximum m and s = sum
// exp(l - m), and the target's logit t.  With M the largest m:  lse = M + log sum s exp(m - M),  loss =
// lse - t.  Where a small vocabulary has few tiles and long sums, the sums are split instead and leave fp32
// parts of the logits, which are added here before the same is done with them.
//
// Statistics are a 16th or a 32nd of what 16-bit logits would be: 8 bytes for 64 or 128 of them.  The join
// of 4096 rows and 32768 words reads 17 MB in 8 us; that of a few rows is a launch's 3 to 4.
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

// To a new maximum; where there is none yet the exponentials are 0.
__device__ __forceinline__ void join_stats(float& top, float& sum, float m, float s) {
  const float t = fmaxf(top, m), base = t == -INFINITY ? 0.0f : t;
  sum = sum * __expf(top - base) + s * __expf(m - base);
  top = t;
}

// lse = M + log sum.  The loss is (M - t) + log sum and not lse - t: where the target is the likeliest word
// its first part is 0, and the loss as exact as the logarithm, not as lse's last bit (2^-20 at 20).
__device__ __forceinline__ void write_loss(const XentJoinParams& p, uint64_t row, int64_t target,
                                           float top, float sum, float hit) {
  const TargetKind kind = target_kind(target, p.ignore, p.vocab);
  const float rest = logf(sum);
  p.lse[row] = top + rest;
  p.loss[row] = kind == kTargetIgnored ? 0.0f
                : kind == kTargetValid ? (top - hit) + rest
                                       : __int_as_float(0x7fffffff);
}

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
  for (uint32_t i = lane; i < p.slots; i += 128u) {
    float2 c[4];
#pragma unroll
    for (uint32_t j = 0; j < 4; ++j)
      c[j] = i + 32u * j < p.slots ? src[i + 32u * j] : make_float2(-INFINITY, 0.0f);
#pragma unroll
    for (uint32_t j = 0; j < 4; ++j) join_stats(top, sum, c[j].x, c[j].y);
  }
#pragma unroll
  for (uint32_t o = 16; o > 0; o /= 2) {
    const float m = __shfl_xor_sync(0xffffffffu, top, o), s = __shfl_xor_sync(0xffffffffu, sum, o);
    join_stats(top, sum, m, s);
  }
  if (lane == 0) write_loss(p, row, target, top, sum, p.hit[row]);
}

// Logits of split sums: parts [splits][part_rows][pitch] (pitch a multiple of 4).
struct LogitParts {
  const float* parts;
  uint64_t stride4;        // float4s between splits
  uint32_t splits, pitch4;

  __device__ void add4(uint32_t row, uint32_t v, float (&l)[4]) const {
    const float4* src = reinterpret_cast<const float4*>(parts) + static_cast<uint64_t>(row) * pitch4 + v;
    l[0] = l[1] = l[2] = l[3] = 0.0f;
#pragma unroll 4
    for (uint32_t s = 0; s < splits; ++s, src += stride4) {
      const float4 c = __ldcg(src);
      l[0] += c.x, l[1] += c.y, l[2] += c.z, l[3] += c.w;
    }
  }
};

// A block of four warps takes a row: a thread every 128th group of four logits.
__global__ void __launch_bounds__(128) xent_rows_kernel(const XentJoinParams p, const LogitParts parts) {
  __shared__ float2 joint[4];
  __shared__ float hit;
  grid_dependency_wait();
  grid_launch_dependents();
  const uint32_t row = blockIdx.x, lane = threadIdx.x & 31u;
  const int64_t target = p.targets[row];
  float top = -INFINITY, sum = 0.0f;
  for (uint32_t v = threadIdx.x; 4u * v < p.vocab; v += 128u) {
    float l[4];
    parts.add4(row, v, l);
    float m = -INFINITY;
#pragma unroll
    for (uint32_t j = 0; j < 4; ++j) {
      if (4u * v + j >= p.vocab) l[j] = -INFINITY;
      if (target == static_cast<int64_t>(4u * v + j)) hit = l[j];
      m = fmaxf(m, l[j]);
    }
    const float base = m == -INFINITY ? 0.0f : m;
    float s = 0.0f;
#pragma unroll
    for (uint32_t j = 0; j < 4; ++j) s += exp2_fast((l[j] - base) * kLog2e);
    join_stats(top, sum, m, s);
  }
#pragma unroll
  for (uint32_t o = 16; o > 0; o /= 2) {
    const float m = __shfl_xor_sync(0xffffffffu, top, o), s = __shfl_xor_sync(0xffffffffu, sum, o);
    join_stats(top, sum, m, s);
  }
  if (lane == 0) joint[threadIdx.x / 32u] = make_float2(top, sum);
  __syncthreads();
  if (threadIdx.x != 0) return;
#pragma unroll
  for (uint32_t w = 1; w < 4; ++w) join_stats(top, sum, joint[w].x, joint[w].y);
  write_loss(p, row, target, top, sum, hit);
}

struct DlogitsParams {
  LogitParts parts;
  RowWeights rows;
  const float* lse;
  void* out;               // [m][pitch_out], pitch_out a multiple of 4
  uint32_t m, n, first_col, pitch_out;
};

// The gradients of logits from their parts, four columns a thread.
template <int DT>
__global__ void __launch_bounds__(256) xent_dlogits_kernel(const DlogitsParams p) {
  __shared__ float tops[8];
  grid_dependency_wait();
  grid_launch_dependents();
  float top = 0.0f;   // the largest |dloss| of all rows
  for (uint32_t r = threadIdx.x; r < p.m; r += 256u) top = fmaxf(top, p.rows.counted(r));
#pragma unroll
  for (uint32_t o = 16; o > 0; o /= 2) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  if ((threadIdx.x & 31u) == 0) tops[threadIdx.x / 32u] = top;
  __syncthreads();
#pragma unroll
  for (uint32_t w = 0; w < 8; ++w) top = fmaxf(top, tops[w]);
  if (blockIdx.x == 0 && threadIdx.x == 0) p.rows.template write_alpha<DT>(top);
  const uint32_t vecs = (p.n + 3u) / 4u;
  const uint64_t total = static_cast<uint64_t>(p.m) * vecs;
  for (uint64_t i = static_cast<uint64_t>(blockIdx.x) * 256u + threadIdx.x; i < total;
       i += static_cast<uint64_t>(gridDim.x) * 256u) {
    const uint32_t row = static_cast<uint32_t>(i / vecs);
    const uint32_t v = static_cast<uint32_t>(i - static_cast<uint64_t>(row) * vecs);
    float l[4];
    p.parts.add4(row, v, l);
    const float lse = p.lse[row], weight = p.rows.template weight<DT>(row, top);
    const int64_t at = p.rows.targets[row] - static_cast<int64_t>(p.first_col + 4u * v);
    uint2 o;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float d = exp2_fast((l[j] - lse) * kLog2e);
      if (at == j) d -= 1.0f;
      l[j] = weight == 0.0f || 4u * v + j >= p.n ? 0.0f : d * weight;
    }
    o.x = pack_out<DT>(__float_as_uint(l[0]), __float_as_uint(l[1]));
    o.y = pack_out<DT>(__float_as_uint(l[2]), __float_as_uint(l[3]));
    *reinterpret_cast<uint2*>(static_cast<char*>(p.out) +
                              (static_cast<uint64_t>(row) * p.pitch_out + 4u * v) * 2u) = o;
  }
}

}  // namespace tg
