// tg_norm_short_kernel.cuh -- layer norm of short rows, forward and backward: rows that a warp holds
// with one 16-byte vector a lane, 256 values of 16 bits or 128 of fp32 (attention heads, small
// models).
//
// L lanes (a power of two) take a row, the warp 32 / L neighbouring rows at once, so that sums cost
// log2 L shuffles and no lane idles that a wider group would leave without values.  The variance is
// the mean square about the row's mean, which is in a register by then.  Nothing is staged: a warp's
// next rows are on their way in registers while it works on the present ones.
// Rows are read and written in accesses of ACCESS bytes, the largest of 16, 4 and a value's size
// that every row start and the row's length are multiples of.
//
// Against the kernels for longer rows, which give a row a whole warp (caches cold, about 4 us of
// launch in each): 30000 rows of 99 bf16 values forward 13 us instead of 31, backward (with its join)
// 21 instead of 39; of 128, 11 instead of 19 and 17 instead of 27; of 256, 15 instead of 17 and 23
// instead of 27; 5 rows the same.  What bounds it is memory latency: 32 warps of 512 bytes (forward)
// or 16 of 2 KiB (backward) in flight an SM.
#pragma once

#include "tg_norm_kernel.cuh"

namespace tg {

constexpr int kShortFwdThreads = 256, kShortFwdCtas = 4;   // of a CTA; CTAs an SM
constexpr int kShortBwdThreads = 512, kShortBwdRows = 2;   // one CTA an SM; rows of a lane a turn

// The first ``left`` (at most kVec<T>) values at p, the others zero; ``left`` is a multiple of the
// values in an access.
template <typename T, int ACCESS>
__device__ __forceinline__ V16 load_part(const char* p, int left) {
  constexpr int kPer = ACCESS / static_cast<int>(sizeof(T));
  V16 r = {{0u, 0u, 0u, 0u}};
  if constexpr (ACCESS == 16) {
    if (left > 0) r = load16(p);
  } else {
#pragma unroll
    for (int j = 0; j < 16 / ACCESS; ++j) {
      if (left <= j * kPer) continue;
      if constexpr (ACCESS == 4)
        r.w[j] = *reinterpret_cast<const uint32_t*>(p + 4 * j);
      else
        r.w[j / 2] |= static_cast<uint32_t>(*reinterpret_cast<const uint16_t*>(p + 2 * j))
                      << (16 * (j & 1));
    }
  }
  return r;
}
template <typename T, int ACCESS>
__device__ __forceinline__ void store_part(char* p, const V16& r, int left) {
  constexpr int kPer = ACCESS / static_cast<int>(sizeof(T));
  if constexpr (ACCESS == 16) {
    if (left > 0) store16(p, r);
  } else {
#pragma unroll
    for (int j = 0; j < 16 / ACCESS; ++j) {
      if (left <= j * kPer) continue;
      if constexpr (ACCESS == 4)
        *reinterpret_cast<uint32_t*>(p + 4 * j) = r.w[j];
      else
        store_one<T>(p, r, j);
    }
  }
}

// Sum over the 2^shift lanes of a row.
__device__ __forceinline__ float row_sum(float v, uint32_t shift) {
#pragma unroll
  for (uint32_t o = 0; o < 5u; ++o)
    if (o < shift) v += __shfl_xor_sync(0xffffffffu, v, 1u << o);
  return v;
}

template <typename TX, typename TP, bool KEEP, int ACCESS>
__global__ void __launch_bounds__(kShortFwdThreads, kShortFwdCtas)
    norm_fwd_short_kernel(const NormFwdParams p, const uint32_t shift) {
  constexpr int N = kVec<TX>;
  const uint32_t lane = threadIdx.x & 31u, warp = threadIdx.x >> 5;
  const uint32_t v = lane & ((1u << shift) - 1u), mine = lane >> shift, per_warp = 32u >> shift;
  const uint32_t col = v * N;
  const int left = values_left<N>(v, p.cols);
  const float cols = static_cast<float>(p.cols);
  grid_dependency_wait();
  grid_launch_dependents();

  float g[N], b[N];
  params_or<TP, N>(p.gamma, col, p.cols, p.wide_params, 1.0f, g);
  params_or<TP, N>(p.beta, col, p.cols, p.wide_params, 0.0f, b);
  const uint64_t step = static_cast<uint64_t>(gridDim.x) * (blockDim.x >> 5) * per_warp;
  uint64_t first = (blockIdx.x + static_cast<uint64_t>(gridDim.x) * warp) * per_warp;
  auto load = [&](uint64_t row) {
    return load_part<TX, ACCESS>(
        p.x.base + static_cast<int64_t>(row) * p.x.pitch + v * 16u, row < p.rows ? left : 0);
  };
  V16 next = load(first + mine);
  for (; first < p.rows; first += step) {
    const uint64_t row = first + mine;
    float x[N];
    values<TX>(next, x);
    next = load(row + step);
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < N; ++i) s += x[i];
    float mean = row_sum(s, shift) / cols;
    float q = 0.0f;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const float d = i < left ? x[i] - mean : 0.0f;
      q = fmaf(d, d, q);
    }
    float square = row_sum(q, shift) / cols;
    // 16-bit values add up exactly over a short row, so equal ones have their value as mean
    if (sizeof(TX) == 4 && __any_sync(0xffffffffu, mean_outweighs(mean, square))) {
      float e = 0.0f;
#pragma unroll
      for (int i = 0; i < N; ++i) e += i < left ? x[i] - mean : 0.0f;
      e = row_sum(e, shift) / cols;
      if (mean_outweighs(mean, square)) correct_mean(mean, square, e);
    }
    const float rstd = inverse_root(square + p.eps);
    const bool valid = row < p.rows;
    if (v == 0u && valid) {
      if (p.mean) p.mean[row] = mean;
      if (p.rstd) p.rstd[row] = rstd;
    }
    float o[N];
#pragma unroll
    for (int i = 0; i < N; ++i) o[i] = fmaf((x[i] - mean) * rstd, g[i], b[i]);
    const V16 out = rounded<TX>(o);
    store_part<TX, ACCESS>(p.y.base + static_cast<int64_t>(row) * p.y.pitch + v * 16u, out,
                           valid ? left : 0);
    if constexpr (KEEP) {
      values<TX>(out, o);   // as rounded
#pragma unroll
      for (int i = 0; i < N; ++i) o[i] = i < left ? o[i] : 0.0f;
      __syncwarp();
      uint32_t k[N / 4];
      const uint32_t scale = ckpt8_quantise<N>(o, k);   // the 32 / N lanes of a block have one row
      if (valid && col < p.blocks * kCkptBlock) {
        const uint64_t block = row * p.blocks + col / kCkptBlock;
        store_kept<N>(p.q + block * kCkptBlock + col % kCkptBlock, k);
        if (col % kCkptBlock == 0) p.s[block] = static_cast<uint8_t>(scale);
      }
    }
  }
}

// Each lane keeps the sums of dy xh and dy of its columns over all its rows.  At the end lanes of
// the same columns are added, then the warps in pairs, always in the same order; the CTA writes one
// row of partial sums for norm_bwd_join_kernel.  blockDim.x is 32 times a power of two.
template <typename TX, typename TP, bool KEPT, int ACCESS>
__global__ void __launch_bounds__(kShortBwdThreads, 1)
    norm_bwd_short_kernel(const NormBwdParams p, const uint32_t shift) {
  constexpr int N = kVec<TX>;
  __shared__ float4 sums[kShortBwdThreads / 64][2][N / 4][32];
  const uint32_t lane = threadIdx.x & 31u, warp = threadIdx.x >> 5;
  const uint32_t v = lane & ((1u << shift) - 1u), mine = lane >> shift, per_warp = 32u >> shift;
  const uint32_t col = v * N;
  const int left = values_left<N>(v, p.cols);
  const float inv_cols = 1.0f / static_cast<float>(p.cols);
  grid_dependency_wait();
  grid_launch_dependents();

  float g[N];
  params_or<TP, N>(p.gamma, col, p.cols, p.wide_params, 1.0f, g);
  const uint64_t step = static_cast<uint64_t>(gridDim.x) * (blockDim.x >> 5) * per_warp;
  uint64_t first = (blockIdx.x + static_cast<uint64_t>(gridDim.x) * warp) * per_warp;
  constexpr int R = kShortBwdRows;
  V16 next_dy[R], next_x[R];   // of a checkpoint: N bytes and the scale
  float next_mean[R], next_rstd[R];
  auto load = [&](uint64_t row, int r) {
    const bool valid = row < p.rows;
    const int n = valid ? left : 0;
    next_dy[r] = load_part<TX, ACCESS>(
        p.dy.base + static_cast<int64_t>(row) * p.dy.pitch + v * 16u, n);
    if constexpr (KEPT) {
      uint32_t q[N / 4] = {}, s = 127u;
      if (n > 0) {
        const uint64_t block = row * p.blocks + col / kCkptBlock;
        load_kept<N>(p.q + block * kCkptBlock + col % kCkptBlock, q);
        s = p.s[block];
      }
      next_x[r] = V16{{q[0], q[N / 4 - 1], 0u, s}};
    } else {
      next_x[r] = load_part<TX, ACCESS>(
          p.x.base + static_cast<int64_t>(row) * p.x.pitch + v * 16u, n);
    }
    next_mean[r] = valid ? p.mean[row] : 0.0f;
    next_rstd[r] = valid ? p.rstd[row] : 0.0f;
  };
  float dg[N], db[N];
#pragma unroll
  for (int i = 0; i < N; ++i) dg[i] = db[i] = 0.0f;
#pragma unroll
  for (int r = 0; r < R; ++r) load(first + mine + r * step, r);
  for (; first < p.rows; first += R * step) {
    float dy[R][N], xh[R][N], rstd[R], s0[R], s1[R];   // s0, s1: sums of dy gamma, and of it times xh
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const float mean = next_mean[r];
      rstd[r] = next_rstd[r];
      values<TX>(next_dy[r], dy[r]);
      if constexpr (KEPT) {
        kept_less<N>(next_x[r].w, next_x[r].w[3], mean, xh[r]);
      } else {
        values<TX>(next_x[r], xh[r]);
#pragma unroll
        for (int i = 0; i < N; ++i) xh[r][i] -= mean;
      }
      load(first + mine + (R + r) * step, r);
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
      s0[r] = s1[r] = 0.0f;
#pragma unroll
      for (int i = 0; i < N; ++i) {
        xh[r][i] = i < left ? xh[r][i] * rstd[r] : 0.0f;
        dg[i] = fmaf(dy[r][i], xh[r][i], dg[i]);
        db[i] += dy[r][i];
        dy[r][i] *= g[i];
        s0[r] += dy[r][i];
        s1[r] = fmaf(dy[r][i], xh[r][i], s1[r]);
      }
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
      s0[r] = row_sum(s0[r], shift);
      s1[r] = row_sum(s1[r], shift);
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {   // dx = rstd gd - rstd c1 - xh rstd c2
      const uint64_t row = first + mine + r * step;
      const float c1 = s0[r] * inv_cols * rstd[r], c2 = s1[r] * inv_cols * rstd[r];
      float dx[N];
#pragma unroll
      for (int i = 0; i < N; ++i) dx[i] = fmaf(-xh[r][i], c2, fmaf(dy[r][i], rstd[r], -c1));
      store_part<TX, ACCESS>(p.dx.base + static_cast<int64_t>(row) * p.dx.pitch + v * 16u,
                             rounded<TX>(dx), row < p.rows ? left : 0);
    }
  }
  if (p.partials == nullptr) return;
  __syncwarp();
#pragma unroll
  for (uint32_t o = 0; o < 5u; ++o) {
    if (o < shift) continue;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      dg[i] += __shfl_xor_sync(0xffffffffu, dg[i], 1u << o);
      db[i] += __shfl_xor_sync(0xffffffffu, db[i], 1u << o);
    }
  }
  for (uint32_t half = blockDim.x >> 6; half > 0u; half >>= 1) {
    if (warp >= half && warp < 2u * half) {
#pragma unroll
      for (int i = 0; i < N; i += 4) {
        sums[warp - half][0][i / 4][lane] = make_float4(dg[i], dg[i + 1], dg[i + 2], dg[i + 3]);
        sums[warp - half][1][i / 4][lane] = make_float4(db[i], db[i + 1], db[i + 2], db[i + 3]);
      }
    }
    __syncthreads();
    if (warp < half) {
#pragma unroll
      for (int i = 0; i < N; i += 4) {
        const float4 a = sums[warp][0][i / 4][lane], b = sums[warp][1][i / 4][lane];
        dg[i] += a.x; dg[i + 1] += a.y; dg[i + 2] += a.z; dg[i + 3] += a.w;
        db[i] += b.x; db[i + 1] += b.y; db[i + 2] += b.z; db[i + 3] += b.w;
      }
    }
    __syncthreads();
  }
  if (warp != 0u || mine != 0u) return;
  float* out = p.partials + static_cast<uint64_t>(blockIdx.x) * 2u * p.part_cols;
#pragma unroll
  for (int i = 0; i < N; i += 4) {
    if (col + i >= p.part_cols) continue;
    *reinterpret_cast<float4*>(out + col + i) =
        make_float4(dg[i], dg[i + 1], dg[i + 2], dg[i + 3]);
    *reinterpret_cast<float4*>(out + p.part_cols + col + i) =
        make_float4(db[i], db[i + 1], db[i + 2], db[i + 3]);
  }
}

}  // namespace tg
