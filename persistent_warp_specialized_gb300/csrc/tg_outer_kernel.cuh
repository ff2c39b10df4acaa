// tg_outer_kernel.cuh -- gradients towards weights from at most 8 rows:
//
//   out[m, n] = alpha sum_t a[t, m] b[t, n]
//
// What bounds it is writing the result, 2 bytes for at most 8 multiplications, so it goes without the tensor
// core, whose tiles would multiply 120 rows of zeros for 8 and whose set-up takes longer than most of
// these products.  a and b come in one or two 16-bit terms, which are added: the sums are fp32's own.
//
// A thread has 8 neighbouring columns of b in registers, all rows of them, and walks down m; the a of
// a block's range of m lie in shared memory as fp32, t next to t, and a warp reads the same ones.
// Measured (bf16, us, with what comes before them; by the pair kernel): 3 rows, 34186 x 1472 44 (62); a gated
// backward pass of 2 rows, 1200 x 5896 16.3 (26.5).
#pragma once

#include "tg_gated_kernel.cuh"

namespace tg {

constexpr uint32_t kOuterCols = 256, kOuterThreads = 256;   // columns of a block; 8 warps, a row of m each
constexpr uint32_t kOuterMostM = 256;

struct OuterParams {
  const void *a, *a_rest;            // [rows][m]; the second term or null
  const void *b[2], *b_rest[2];      // [rows][n] of each result (blockIdx.z)
  void* out[2];
  int64_t ld_a, ld_b, ld_out[2];
  uint32_t rows, m, n;
  uint32_t block_m;                  // rows of m of a block
  const float* alpha;
};

// 8 values of a row at ``at`` (16-byte aligned), of both terms
template <int DT>
__device__ __forceinline__ void add8(const uint4& w, float (&v)[8]) {
  const uint32_t words[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float2 f = unpack_in<DT>(words[j]);
    v[2 * j] += f.x;
    v[2 * j + 1] += f.y;
  }
}
__device__ __forceinline__ uint4 load8(const void* base, int64_t at, bool in) {
  return base != nullptr && in
             ? *reinterpret_cast<const uint4*>(static_cast<const char*>(base) + 2 * at)
             : make_uint4(0u, 0u, 0u, 0u);
}

// T: rows, rounded up to a power of two.  a's rows may be read up to the next multiple of 8 values.
template <int DT, int T>
__global__ void __launch_bounds__(kOuterThreads) outer_kernel(const __grid_constant__ OuterParams p) {
  __shared__ __align__(16) float a[kOuterMostM * T];
  grid_dependency_wait();
  grid_launch_dependents();
  const uint32_t z = blockIdx.z, m0 = blockIdx.y * p.block_m;
  const uint32_t ms = min(p.block_m, p.m - m0);
  const uint32_t lane = threadIdx.x & 31u, n = blockIdx.x * kOuterCols + 8u * lane;
  const bool in = n < p.n;
  // all of b's loads, and then all of a's, are under way before the first is used
  uint4 w[T], w_rest[T];
#pragma unroll
  for (uint32_t t = 0; t < T; ++t) {
    w[t] = load8(p.b[z], t * p.ld_b + n, in && t < p.rows);
    w_rest[t] = load8(p.b_rest[z], t * p.ld_b + n, in && t < p.rows);
  }
  constexpr uint32_t kMostVecs = (kOuterMostM * T / 8 + kOuterThreads - 1) / kOuterThreads;
  const uint32_t vecs = p.block_m / 8u;
#pragma unroll
  for (uint32_t k = 0; k < kMostVecs; ++k) {
    const uint32_t i = threadIdx.x + k * kOuterThreads, t = i / vecs, m = (i - t * vecs) * 8u;
    if (t >= T) break;
    const bool is = t < p.rows && m < ms;
    float v[8] = {};
    const uint4 x = load8(p.a, t * p.ld_a + m0 + m, is), y = load8(p.a_rest, t * p.ld_a + m0 + m, is);
    add8<DT>(x, v);
    add8<DT>(y, v);
#pragma unroll
    for (uint32_t j = 0; j < 8; ++j) a[(m + j) * T + t] = v[j];
  }
  float b[T][8];
#pragma unroll
  for (uint32_t t = 0; t < T; ++t) {
#pragma unroll
    for (int j = 0; j < 8; ++j) b[t][j] = 0.0f;
    add8<DT>(w[t], b[t]);
    add8<DT>(w_rest[t], b[t]);
  }
  const float alpha = p.alpha ? *p.alpha : 1.0f;
  __syncthreads();
  if (!in) return;
  char* out = static_cast<char*>(p.out[z]) + 2 * n;
  for (uint32_t m = threadIdx.x / 32u; m < ms; m += kOuterThreads / 32u) {
    float s[8] = {};
#pragma unroll
    for (uint32_t t = 0; t < T; ++t) {
      const float x = a[m * T + t];
#pragma unroll
      for (int j = 0; j < 8; ++j) s[j] = fmaf(x, b[t][j], s[j]);
    }
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
      w[j] = pack_out<DT>(__float_as_uint(s[2 * j] * alpha), __float_as_uint(s[2 * j + 1] * alpha));
    st_global_v4(out + (static_cast<int64_t>(m0) + m) * p.ld_out[z] * 2, w[0], w[1], w[2], w[3]);
  }
}

}  // namespace tg
