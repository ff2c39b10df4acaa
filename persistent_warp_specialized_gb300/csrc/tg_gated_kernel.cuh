// tg_gated_kernel.cuh -- what the gated feed-forward projections do outside the tensor core:
//
//   the backward pass of h = act(g) u:   dg = dh u act'(g),   du = dh act(g)
//   and h from partial sums of g and u when K was split.
//
// Both are bound by memory: 8 values a thread and tensor in one 16-byte access each, two vectors ahead.
//
// fp16 has few exponents, and dg and du are products of three values: they may leave its range at either
// end where the gradients that are made of them do not (dh of 2e-5 and u of 0.05: gradients 1.3e-3 off,
// where a rounding makes 2e-4; dh of 8e3 and u of 20: no number at all).  So they are held times a power of two,
// which the products' alpha undoes.  The first pass takes 2^4 and finds the largest; where that does not lie in
// [4, 65504] then, which gradients of a scaled loss seldom miss, a second pass makes them again with the
// power of two that takes the largest to 2^14 .. 2^15.  Steps are so at most 2^-26 of the largest value.  Measured
// (fp16, whole backward pass, us; before / guess right / made again): 333 x 1000 x 2008 19.6 / 22.8 / 24.8,
// 2048 x 2048 x 5632 131 / 136 / 152, 8192 x 4096 x 8192 1462 / 1436 / 1585.
// Measured (bf16, 4096 x 8192, 336 MB read and written): SiLU 51 us, 6.5 TB/s; GELU 56, of which issuing
// its instructions takes 68 % of the slots.
#pragma once

#include "tg_linear_kernel.cuh"

namespace tg {

template <int DT>
__device__ __forceinline__ float2 unpack_in(uint32_t w) {
  if constexpr (DT == 1) {
    return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&w));
  } else {
    return __half22float2(*reinterpret_cast<const __half2*>(&w));
  }
}

struct GatedGradParams {
  const void *dh, *g, *u;
  void* dgu;                       // [rows][2 vecs x 8]: dg, then du
  void* rest;                      // TWO: the same of what rounding them left
  int64_t ld_dh, ld_g, ld_u;       // elements
  uint32_t rows, vecs;             // vectors of 8 values in a row
  uint32_t act;
  float* tops;                     // fp16: each block's largest |dg|, |du| that is finite
  float* alpha;                    // fp16: what undoes the scale
};

constexpr int kGradGuess = 4;      // fp16: the first pass's power of two

// The power of two for gradients of at most ``top``.
__device__ __forceinline__ int grad_exponent(float top) {
  const float guess = top * (1 << kGradGuess);
  if (top == 0.0f || (guess >= 4.0f && guess <= 65504.0f)) return kGradGuess;
  const int e = static_cast<int>(__float_as_uint(top) >> 23) - 127;   // top in 2^e .. 2^(e + 1)
  return max(-30, min(14 - e, 60));   // |dg| < 2^33; past 2^-46 nothing is left in fp16 anyway
}
__device__ __forceinline__ float power_of_2(int e) { return __int_as_float((e + 127) << 23); }

// The largest of a block's 256 threads' values, in every thread.
__device__ __forceinline__ float block_top(float v) {
  __shared__ float warps[8];
#pragma unroll
  for (uint32_t o = 16; o > 0; o /= 2) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  if ((threadIdx.x & 31u) == 0) warps[threadIdx.x / 32u] = v;
  __syncthreads();
#pragma unroll
  for (uint32_t w = 0; w < 8; ++w) v = fmaxf(v, warps[w]);
  return v;
}

// A thread takes every so many'th vector of the matrix, two at a time.
// TWO: in two terms.  AGAIN: the second pass in fp16, by as many blocks as the first.
template <int DT, bool TWO, bool AGAIN>
__global__ void __launch_bounds__(256) gated_grad_kernel(const GatedGradParams p) {
  static_assert(DT == 0 || !AGAIN, "bf16 has fp32's exponents");
  grid_dependency_wait();
  grid_launch_dependents();
  float factor = power_of_2(kGradGuess), top = 0.0f;
  if constexpr (AGAIN) {
    for (uint32_t i = threadIdx.x; i < gridDim.x; i += 256u) top = fmaxf(top, __ldcg(p.tops + i));
    const int e = grad_exponent(block_top(top));
    if (blockIdx.x == 0 && threadIdx.x == 0) *p.alpha = power_of_2(-e);
    if (e == kGradGuess) return;
    factor = power_of_2(e);
  }
  const uint64_t total = static_cast<uint64_t>(p.rows) * p.vecs;
  const uint64_t stride = static_cast<uint64_t>(gridDim.x) * blockDim.x;
  auto at = [](const void* base, uint64_t row, int64_t ld, uint32_t v) {
    return reinterpret_cast<const uint4*>(static_cast<const char*>(base) +
                                          (static_cast<int64_t>(row) * ld + 8ll * v) * 2);
  };
  auto work = [&](uint64_t row, uint32_t v, const uint4& dh4, const uint4& g4, const uint4& u4) {
    const uint32_t dhw[4] = {dh4.x, dh4.y, dh4.z, dh4.w}, gw[4] = {g4.x, g4.y, g4.z, g4.w},
                   uw[4] = {u4.x, u4.y, u4.z, u4.w};
    uint32_t dgw[4], duw[4], dg_rest[4], du_rest[4];
    auto pack = [&](float x, float y, uint32_t& rest) {
      if constexpr (DT == 0) {
        if constexpr (!AGAIN) {
          top = fmaxf(top, fabsf(x) < INFINITY ? fabsf(x) : 0.0f);
          top = fmaxf(top, fabsf(y) < INFINITY ? fabsf(y) : 0.0f);
        }
        x *= factor;
        y *= factor;
      }
      const uint32_t w = pack_out<DT>(__float_as_uint(x), __float_as_uint(y));
      if constexpr (TWO) {
        const float2 back = unpack_in<DT>(w);
        rest = pack_out<DT>(__float_as_uint(left_over(x, back.x)),
                            __float_as_uint(left_over(y, back.y)));
      }
      return w;
    };
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 dh = unpack_in<DT>(dhw[i]), g = unpack_in<DT>(gw[i]), u = unpack_in<DT>(uw[i]);
      const Gate a = gate_of(g.x, p.act), b = gate_of(g.y, p.act);
      const float ax = g.x * a.s, bx = g.y * b.s;
      dgw[i] = pack(dh.x * u.x * fmaf(ax * (1.0f - a.s), a.slope, a.s),
                    dh.y * u.y * fmaf(bx * (1.0f - b.s), b.slope, b.s), dg_rest[i]);
      duw[i] = pack(dh.x * ax, dh.y * bx, du_rest[i]);
    }
    const uint64_t at = (row * 2u * p.vecs + v) * 16u, next = static_cast<uint64_t>(p.vecs) * 16u;
    char* to = static_cast<char*>(p.dgu) + at;
    st_global_v4(to, dgw[0], dgw[1], dgw[2], dgw[3]);
    st_global_v4(to + next, duw[0], duw[1], duw[2], duw[3]);
    if constexpr (TWO) {
      to = static_cast<char*>(p.rest) + at;
      st_global_v4(to, dg_rest[0], dg_rest[1], dg_rest[2], dg_rest[3]);
      st_global_v4(to + next, du_rest[0], du_rest[1], du_rest[2], du_rest[3]);
    }
  };
  for (uint64_t i = static_cast<uint64_t>(blockIdx.x) * blockDim.x + threadIdx.x; i < total;
       i += 2u * stride) {
    const uint64_t i1 = i + stride;
    const bool two = i1 < total;
    const uint64_t r0 = i / p.vecs, r1 = two ? i1 / p.vecs : r0;
    const uint32_t v0 = static_cast<uint32_t>(i - r0 * p.vecs);
    const uint32_t v1 = two ? static_cast<uint32_t>(i1 - r1 * p.vecs) : v0;
    const uint4 dh0 = __ldcs(at(p.dh, r0, p.ld_dh, v0)), g0 = __ldcs(at(p.g, r0, p.ld_g, v0)),
                u0 = __ldcs(at(p.u, r0, p.ld_u, v0));
    uint4 dh1 = dh0, g1 = g0, u1 = u0;
    if (two) {
      dh1 = __ldcs(at(p.dh, r1, p.ld_dh, v1));
      g1 = __ldcs(at(p.g, r1, p.ld_g, v1));
      u1 = __ldcs(at(p.u, r1, p.ld_u, v1));
    }
    work(r0, v0, dh0, g0, u0);
    if (two) work(r1, v1, dh1, g1, u1);
  }
  if constexpr (DT == 0 && !AGAIN) {
    top = block_top(top);
    if (threadIdx.x == 0) p.tops[blockIdx.x] = top;
  }
}

struct GatedJoinParams {
  const float *g_parts, *u_parts;
  uint64_t split_stride;           // values between splits
  uint32_t splits, rows, outs;
  uint32_t act;
  void *h, *g, *u;                 // g and u together, or neither
  int64_t ld_h, ld_g, ld_u;
};

// A thread takes 4 neighbouring columns and adds the splits in order.
template <int DT>
__global__ void __launch_bounds__(256) gated_join_kernel(const GatedJoinParams p) {
  grid_dependency_wait();
  grid_launch_dependents();
  const uint32_t vecs = p.outs / 4u;
  const uint64_t total = static_cast<uint64_t>(p.rows) * vecs, stride4 = p.split_stride / 4u;
  for (uint64_t i = static_cast<uint64_t>(blockIdx.x) * blockDim.x + threadIdx.x; i < total;
       i += static_cast<uint64_t>(gridDim.x) * blockDim.x) {
    const uint64_t row = i / vecs;
    const uint32_t v = static_cast<uint32_t>(i - row * vecs);
    float g[4] = {}, u[4] = {};
#pragma unroll 4
    for (uint32_t s = 0; s < p.splits; ++s) {
      const float4 a = __ldcg(reinterpret_cast<const float4*>(p.g_parts) + i + s * stride4);
      const float4 b = __ldcg(reinterpret_cast<const float4*>(p.u_parts) + i + s * stride4);
      g[0] += a.x, g[1] += a.y, g[2] += a.z, g[3] += a.w;
      u[0] += b.x, u[1] += b.y, u[2] += b.z, u[3] += b.w;
    }
    auto put = [&](void* base, int64_t ld, const float (&f)[4]) {
      uint2 o;
      o.x = pack_out<DT>(__float_as_uint(f[0]), __float_as_uint(f[1]));
      o.y = pack_out<DT>(__float_as_uint(f[2]), __float_as_uint(f[3]));
      *reinterpret_cast<uint2*>(static_cast<char*>(base) +
                                (static_cast<int64_t>(row) * ld + 4ll * v) * 2) = o;
    };
    if (p.g != nullptr) {
      put(p.g, p.ld_g, g);
      put(p.u, p.ld_u, u);
    }
    float h[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) h[j] = g[j] * gate_of(g[j], p.act).s * u[j];
    put(p.h, p.ld_h, h);
  }
}

}  // namespace tg
