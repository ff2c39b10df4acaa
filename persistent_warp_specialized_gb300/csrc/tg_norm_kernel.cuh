// tg_norm_kernel.cuh -- layer norm over the rows of x [rows, cols], forward and backward.
//
// Forward, in 32 bits:  mean = sum x / cols,  rstd = 1 / sqrt(sum (x - mean)^2 / cols + eps),
// y = (x - mean) rstd gamma + beta, rounded once; optionally the 8-bit checkpoint of the rounded y
// as well (tg_rows.cuh), so that it need not be read again to be packed.
// Backward, with xh = (x - mean) rstd and g = dy gamma:
//   dx = rstd (g - sum g / cols - xh sum (g xh) / cols),  dgamma = sum_rows dy xh,
//   dbeta = sum_rows dy;  x is the tensor, or its 8-bit checkpoint.
// Both are bound by memory: a row stays in registers from its one read to the result's write.
//
// The variance is the sum of squares about the mean in two steps that need one exchange between
// warps: each warp takes the mean of its own values and their squares about that mean, and
// sum (x - mean)^2 = sum over warps of [M2_w + n_w (mean_w - mean)^2].  No difference of large
// sums is formed, so a large mean costs no digits.
#pragma once

#include "tg_rows.cuh"

namespace tg {

struct NormFwdParams {
  const void* x;
  const void* gamma;   // may be null (ones)
  const void* beta;    // may be null (zeros)
  void* y;
  float* mean;         // may be null
  float* rstd;         // may be null
  uint8_t* q;          // checkpoint of y (KEEP)
  uint8_t* s;
  uint32_t rows, cols, blocks;
  int64_t ld_x, ld_y;
  float eps;
};

// What one warp of a row's G threads holds of the row: vectors (k G + 32 w) .. + 32 for each k.
template <int VE>
__device__ __forceinline__ float warp_share(uint32_t g_threads, uint32_t w, int items,
                                            uint32_t cols) {
  uint32_t n = 0;
  for (int k = 0; k < items; ++k) {
    const uint32_t at = (k * g_threads + 32u * w) * VE;
    n += at >= cols ? 0u : (cols - at < 32u * VE ? cols - at : 32u * VE);
  }
  return static_cast<float>(n);
}

// y of VE values (and their checkpoint); ``col`` may lie past the row's end, all lanes call it.
template <typename TX, typename TP, int VE, bool KEEP>
__device__ __forceinline__ void norm_write(const NormFwdParams& p, uint32_t row, uint32_t col,
                                           const float (&v)[VE], float mean, float rstd) {
  const int64_t left = static_cast<int64_t>(p.cols) - col;
  Raw<TX, VE> out;
  float g[VE], b[VE];
#pragma unroll
  for (int i = 0; i < VE; ++i) g[i] = 1.0f, b[i] = 0.0f;
  if (p.gamma) {
    const Raw<TP, VE> r = load_some<TP, VE>(static_cast<const TP*>(p.gamma) + col, left);
#pragma unroll
    for (int i = 0; i < VE; ++i) g[i] = to_f32(r.v[i]);
  }
  if (p.beta) {
    const Raw<TP, VE> r = load_some<TP, VE>(static_cast<const TP*>(p.beta) + col, left);
#pragma unroll
    for (int i = 0; i < VE; ++i) b[i] = to_f32(r.v[i]);
  }
#pragma unroll
  for (int i = 0; i < VE; ++i) out.v[i] = from_f32<TX>(fmaf((v[i] - mean) * rstd, g[i], b[i]));
  store_some<TX, VE>(static_cast<TX*>(p.y) + static_cast<int64_t>(row) * p.ld_y + col, out, left);
  if constexpr (KEEP) {
    float o[VE];
#pragma unroll
    for (int i = 0; i < VE; ++i) o[i] = i < left ? to_f32(out.v[i]) : 0.0f;
    Raw<uint8_t, VE> q;
    const uint32_t s = ckpt8_quantise<VE>(o, q);
    const uint32_t b32 = col / kCkptBlock;
    if (b32 < p.blocks) {
      const uint64_t block = static_cast<uint64_t>(row) * p.blocks + b32;
      *reinterpret_cast<Raw<uint8_t, VE>*>(p.q + block * kCkptBlock + col % kCkptBlock) = q;
      if (col % kCkptBlock == 0) p.s[block] = static_cast<uint8_t>(s);
    }
  }
}

// A row in the registers of G threads: a warp (WARP_ROW, several rows per CTA), or the CTA.  Thread
// t holds vectors t, t + G, ... of VE values, ITEMS of them, so G * ITEMS * VE >= cols.
template <typename TX, typename TP, int VE, int ITEMS, bool WARP_ROW, bool KEEP>
__global__ void __launch_bounds__(WARP_ROW ? 128 : 1024) norm_fwd_kernel(const NormFwdParams p) {
  __shared__ float2 part[32];
  const uint32_t lane = threadIdx.x & 31u, warp = threadIdx.x >> 5;
  const uint32_t g_threads = WARP_ROW ? 32u : blockDim.x;
  const uint32_t t = WARP_ROW ? lane : threadIdx.x;
  const uint32_t row = WARP_ROW ? blockIdx.x * (blockDim.x >> 5) + warp : blockIdx.x;
  grid_dependency_wait();
  grid_launch_dependents();
  if (row >= p.rows) return;   // whole warps (WARP_ROW), never part of a CTA otherwise
  const TX* x = static_cast<const TX*>(p.x) + static_cast<int64_t>(row) * p.ld_x;
  float v[ITEMS][VE];
#pragma unroll
  for (int k = 0; k < ITEMS; ++k) {
    const uint32_t col = (k * g_threads + t) * VE;
    const Raw<TX, VE> r = load_some<TX, VE>(x + col, static_cast<int64_t>(p.cols) - col);
#pragma unroll
    for (int i = 0; i < VE; ++i) v[k][i] = to_f32(r.v[i]);
  }
  float sum = 0.0f;
#pragma unroll
  for (int k = 0; k < ITEMS; ++k)
#pragma unroll
    for (int i = 0; i < VE; ++i) sum += v[k][i];   // values past the end are zero
  sum = warp_sum(sum);
  const uint32_t w = WARP_ROW ? 0u : warp;
  const float n = warp_share<VE>(g_threads, w, ITEMS, p.cols);
  const float m = n > 0.0f ? sum / n : 0.0f;
  float m2 = 0.0f;
#pragma unroll
  for (int k = 0; k < ITEMS; ++k) {
    const int64_t left = static_cast<int64_t>(p.cols) - (k * g_threads + t) * VE;
#pragma unroll
    for (int i = 0; i < VE; ++i) {
      const float d = v[k][i] - m;
      m2 += i < left ? d * d : 0.0f;
    }
  }
  m2 = warp_sum(m2);
  float mean = m;
  if constexpr (!WARP_ROW) {
    const uint32_t warps = blockDim.x >> 5;
    if (lane == 0) part[warp] = make_float2(sum, m2);
    __syncthreads();
    const float2 mine = lane < warps ? part[lane] : make_float2(0.0f, 0.0f);
    mean = warp_sum(mine.x) / static_cast<float>(p.cols);
    const float nl = lane < warps ? warp_share<VE>(g_threads, lane, ITEMS, p.cols) : 0.0f;
    const float d = nl > 0.0f ? mine.x / nl - mean : 0.0f;
    m2 = warp_sum(mine.y + nl * d * d);
  }
  const float rstd = 1.0f / sqrtf(m2 / static_cast<float>(p.cols) + p.eps);
  if (t == 0) {
    if (p.mean) p.mean[row] = mean;
    if (p.rstd) p.rstd[row] = rstd;
  }
#pragma unroll
  for (int k = 0; k < ITEMS; ++k)
    norm_write<TX, TP, VE, KEEP>(p, row, (k * g_threads + t) * VE, v[k], mean, rstd);
}

// Any width: the CTA walks its row three times; the second and third reads come from the L2.
template <typename TX, typename TP, int VE, bool KEEP>
__global__ void __launch_bounds__(1024) norm_fwd_long_kernel(const NormFwdParams p) {
  __shared__ float part[2][32];
  const uint32_t lane = threadIdx.x & 31u, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  grid_dependency_wait();
  grid_launch_dependents();
  const uint32_t row = blockIdx.x;
  const TX* x = static_cast<const TX*>(p.x) + static_cast<int64_t>(row) * p.ld_x;
  const uint32_t vecs = (p.cols + VE - 1) / VE;
  float stat[2] = {0.0f, 0.0f};   // mean, then sum of squares about it
#pragma unroll 1
  for (int pass = 0; pass < 2; ++pass) {
    float a = 0.0f;
    for (uint32_t j = threadIdx.x; j < vecs; j += blockDim.x) {
      const int64_t left = static_cast<int64_t>(p.cols) - static_cast<int64_t>(j) * VE;
      const Raw<TX, VE> r = load_some<TX, VE>(x + static_cast<int64_t>(j) * VE, left);
#pragma unroll
      for (int i = 0; i < VE; ++i) {
        const float d = to_f32(r.v[i]) - stat[0];
        a += i < left ? (pass ? d * d : d) : 0.0f;
      }
    }
    a = warp_sum(a);
    if (lane == 0) part[pass][warp] = a;
    __syncthreads();
    a = warp_sum(lane < warps ? part[pass][lane] : 0.0f);
    stat[pass] = a / static_cast<float>(p.cols);
  }
  const float mean = stat[0], rstd = 1.0f / sqrtf(stat[1] + p.eps);
  if (threadIdx.x == 0) {
    if (p.mean) p.mean[row] = mean;
    if (p.rstd) p.rstd[row] = rstd;
  }
  const uint32_t end = (vecs + 31u) & ~31u;   // whole warps, for the checkpoint's shuffles
  for (uint32_t j = threadIdx.x; j < end; j += blockDim.x) {
    const int64_t left = static_cast<int64_t>(p.cols) - static_cast<int64_t>(j) * VE;
    const Raw<TX, VE> r = load_some<TX, VE>(x + static_cast<int64_t>(j) * VE, left);
    float v[VE];
#pragma unroll
    for (int i = 0; i < VE; ++i) v[i] = to_f32(r.v[i]);
    norm_write<TX, TP, VE, KEEP>(p, row, j * VE, v, mean, rstd);
  }
}

// ---------------------------------------------------------------- backward
struct NormBwdParams {
  const void* dy;
  const void* x;         // the tensor, or (KEPT) null
  const uint8_t* q;      // the checkpoint of x (KEPT)
  const uint8_t* s;
  const void* gamma;     // may be null (ones)
  const float* mean;
  const float* rstd;
  void* dx;
  float* partials;       // [parts][2][cols] sums of dy xh and of dy; null: not wanted
  uint32_t rows, cols, blocks;
  int64_t ld_dy, ld_x, ld_dx;
};

// Where a row's x comes from: VE values at ``col``, as they lie in memory.
template <typename TX, int VE, bool KEPT>
struct XSource {
  using Held = Raw<TX, VE>;
  static __device__ __forceinline__ Held load(const NormBwdParams& p, uint32_t row, uint32_t col,
                                              int64_t left) {
    return load_some<TX, VE>(
        static_cast<const TX*>(p.x) + static_cast<int64_t>(row) * p.ld_x + col, left);
  }
  static __device__ __forceinline__ void values(const Held& h, float (&v)[VE]) {
#pragma unroll
    for (int i = 0; i < VE; ++i) v[i] = to_f32(h.v[i]);
  }
};
template <typename TX, int VE>
struct XSource<TX, VE, true> {
  using Held = Kept<VE>;
  static __device__ __forceinline__ Held load(const NormBwdParams& p, uint32_t row, uint32_t col,
                                              int64_t left) {
    Held h = {};
    if (left > 0) {
      const uint64_t block = static_cast<uint64_t>(row) * p.blocks + col / kCkptBlock;
      h.q = load_raw<uint8_t, VE>(p.q + block * kCkptBlock + col % kCkptBlock);
      h.s = p.s[block];
    }
    return h;
  }
  static __device__ __forceinline__ void values(const Held& h, float (&v)[VE]) {
    kept_values<VE>(h, v);
  }
};

// Rows go to groups of G threads (a CTA holds blockDim.x / G of them, G a multiple of 32), each
// thread keeping the sums of dy xh and dy of its own columns in registers over all its rows.  The
// next row is read while the present one is reduced.  At the end the groups of a CTA add up, and
// the CTA writes one row of partial sums; norm_bwd_join_kernel adds those in a fixed order, so the
// result does not depend on timing.
template <typename TX, typename TP, int VE, int ITEMS, bool KEPT>
__global__ void __launch_bounds__(512) norm_bwd_kernel(const NormBwdParams p, uint32_t g_threads) {
  extern __shared__ float shared_cols[];    // [2][cols], used when a CTA holds several groups
  __shared__ float2 part[2][16];
  using X = XSource<TX, VE, KEPT>;
  const uint32_t lane = threadIdx.x & 31u, warp = threadIdx.x >> 5;
  const uint32_t groups = blockDim.x / g_threads, group = threadIdx.x / g_threads;
  const uint32_t t = threadIdx.x - group * g_threads;
  const uint32_t g_warps = g_threads >> 5, first_warp = group * g_warps;
  grid_dependency_wait();
  grid_launch_dependents();
  float gamma[ITEMS][VE], dg[ITEMS][VE], db[ITEMS][VE];
#pragma unroll
  for (int k = 0; k < ITEMS; ++k) {
    const uint32_t col = (k * g_threads + t) * VE;
#pragma unroll
    for (int i = 0; i < VE; ++i) gamma[k][i] = 1.0f, dg[k][i] = 0.0f, db[k][i] = 0.0f;
    if (p.gamma) {
      const Raw<TP, VE> r = load_some<TP, VE>(static_cast<const TP*>(p.gamma) + col,
                                              static_cast<int64_t>(p.cols) - col);
#pragma unroll
      for (int i = 0; i < VE; ++i) gamma[k][i] = to_f32(r.v[i]);
    }
  }
  const float inv_cols = 1.0f / static_cast<float>(p.cols);
  const uint32_t step = gridDim.x * groups;
  uint32_t row = blockIdx.x * groups + group;
  typename X::Held xr[ITEMS];
  Raw<TX, VE> dyr[ITEMS];
  float mean = 0.0f, rstd = 0.0f;
  auto fetch = [&](uint32_t r) {
#pragma unroll
    for (int k = 0; k < ITEMS; ++k) {
      const uint32_t col = (k * g_threads + t) * VE;
      const int64_t left = static_cast<int64_t>(p.cols) - col;
      xr[k] = X::load(p, r, col, left);
      dyr[k] = load_some<TX, VE>(
          static_cast<const TX*>(p.dy) + static_cast<int64_t>(r) * p.ld_dy + col, left);
    }
    mean = p.mean[r];
    rstd = p.rstd[r];
  };
  if (row < p.rows) fetch(row);
  uint32_t turn = 0;
  while (row < p.rows) {
    float dy[ITEMS][VE], xh[ITEMS][VE];
    float s1 = 0.0f, s2 = 0.0f;
#pragma unroll
    for (int k = 0; k < ITEMS; ++k) {
      const int64_t left = static_cast<int64_t>(p.cols) - (k * g_threads + t) * VE;
      float xv[VE];
      X::values(xr[k], xv);
#pragma unroll
      for (int i = 0; i < VE; ++i) {
        dy[k][i] = to_f32(dyr[k].v[i]);             // zero past the row's end
        xh[k][i] = i < left ? (xv[i] - mean) * rstd : 0.0f;
        const float g = dy[k][i] * gamma[k][i];
        s1 += g;
        s2 = fmaf(g, xh[k][i], s2);
      }
    }
    const float scale = rstd;
    const uint32_t here = row;
    row += step;
    if (row < p.rows) fetch(row);
    s1 = warp_sum(s1);
    s2 = warp_sum(s2);
    if (g_warps > 1) {
      if (lane == 0) part[turn & 1u][warp] = make_float2(s1, s2);
      // the group's own barrier: other groups of the CTA are on other rows
      asm volatile("bar.sync %0, %1;" ::"r"(group + 1u), "r"(g_threads) : "memory");
      const float2 mine =
          lane < g_warps ? part[turn & 1u][first_warp + lane] : make_float2(0.0f, 0.0f);
      s1 = warp_sum(mine.x);
      s2 = warp_sum(mine.y);
      ++turn;   // the other half of ``part``: a slower warp may still read this one
    }
    const float c1 = s1 * inv_cols, c2 = s2 * inv_cols;
#pragma unroll
    for (int k = 0; k < ITEMS; ++k) {
      const uint32_t col = (k * g_threads + t) * VE;
      Raw<TX, VE> out;
#pragma unroll
      for (int i = 0; i < VE; ++i) {
        dg[k][i] = fmaf(dy[k][i], xh[k][i], dg[k][i]);
        db[k][i] += dy[k][i];
        out.v[i] = from_f32<TX>(scale * (fmaf(dy[k][i], gamma[k][i], -c1) - xh[k][i] * c2));
      }
      store_some<TX, VE>(static_cast<TX*>(p.dx) + static_cast<int64_t>(here) * p.ld_dx + col, out,
                         static_cast<int64_t>(p.cols) - col);
    }
  }
  if (p.partials == nullptr) return;
  float* mine = p.partials + static_cast<uint64_t>(blockIdx.x) * 2u * p.cols;
  for (uint32_t turn_of = 0; turn_of < groups; ++turn_of) {   // the groups add up one by one
    if (group == turn_of) {
      const bool first = turn_of == 0, last = turn_of + 1 == groups;
#pragma unroll
      for (int k = 0; k < ITEMS; ++k) {
#pragma unroll
        for (int i = 0; i < VE; ++i) {
          const uint32_t col = (k * g_threads + t) * VE + i;
          if (col >= p.cols) continue;
          float a = dg[k][i], b = db[k][i];
          if (!first) a += shared_cols[col], b += shared_cols[p.cols + col];
          if (last) {
            mine[col] = a;
            mine[p.cols + col] = b;
          } else {
            shared_cols[col] = a;
            shared_cols[p.cols + col] = b;
          }
        }
      }
    }
    if (turn_of + 1 < groups) __syncthreads();
  }
}

// Any width: a CTA walks its row twice (sums, then dx; the second read comes from the L2), and
// norm_bwd_cols_kernel reads x and dy once more for the sums over rows.
template <typename TX, typename TP, int VE, bool KEPT>
__global__ void __launch_bounds__(1024) norm_bwd_long_kernel(const NormBwdParams p) {
  __shared__ float2 part[32];
  using X = XSource<TX, VE, KEPT>;
  const uint32_t lane = threadIdx.x & 31u, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  grid_dependency_wait();
  grid_launch_dependents();
  const uint32_t row = blockIdx.x;
  const float mean = p.mean[row], rstd = p.rstd[row];
  const uint32_t vecs = (p.cols + VE - 1) / VE;
  float c1 = 0.0f, c2 = 0.0f;
#pragma unroll 1
  for (int pass = 0; pass < 2; ++pass) {
    for (uint32_t j = threadIdx.x; j < vecs; j += blockDim.x) {
      const uint32_t col = j * VE;
      const int64_t left = static_cast<int64_t>(p.cols) - col;
      const typename X::Held h = X::load(p, row, col, left);
      const Raw<TX, VE> d = load_some<TX, VE>(
          static_cast<const TX*>(p.dy) + static_cast<int64_t>(row) * p.ld_dy + col, left);
      float xv[VE], gamma[VE];
      X::values(h, xv);
#pragma unroll
      for (int i = 0; i < VE; ++i) gamma[i] = 1.0f;
      if (p.gamma) {
        const Raw<TP, VE> r = load_some<TP, VE>(static_cast<const TP*>(p.gamma) + col, left);
#pragma unroll
        for (int i = 0; i < VE; ++i) gamma[i] = to_f32(r.v[i]);
      }
      Raw<TX, VE> out;
#pragma unroll
      for (int i = 0; i < VE; ++i) {
        const float dy = to_f32(d.v[i]);
        const float xh = i < left ? (xv[i] - mean) * rstd : 0.0f;
        if (pass == 0) {
          c1 = fmaf(dy, gamma[i], c1);
          c2 = fmaf(dy * gamma[i], xh, c2);
        } else {
          out.v[i] = from_f32<TX>(rstd * (fmaf(dy, gamma[i], -c1) - xh * c2));
        }
      }
      if (pass == 1)
        store_some<TX, VE>(static_cast<TX*>(p.dx) + static_cast<int64_t>(row) * p.ld_dx + col, out,
                           left);
    }
    if (pass == 0) {
      c1 = warp_sum(c1);
      c2 = warp_sum(c2);
      if (lane == 0) part[warp] = make_float2(c1, c2);
      __syncthreads();
      const float2 mine = lane < warps ? part[lane] : make_float2(0.0f, 0.0f);
      c1 = warp_sum(mine.x) / static_cast<float>(p.cols);
      c2 = warp_sum(mine.y) / static_cast<float>(p.cols);
    }
  }
}

// Sums over rows for any width: thread t of block (i, j) takes VE columns and rows j, j + parts, ...
template <typename TX, int VE, bool KEPT>
__global__ void __launch_bounds__(128) norm_bwd_cols_kernel(const NormBwdParams p) {
  using X = XSource<TX, VE, KEPT>;
  grid_dependency_wait();
  grid_launch_dependents();
  const uint64_t at = (static_cast<uint64_t>(blockIdx.x) * blockDim.x + threadIdx.x) * VE;
  if (at >= p.cols) return;
  const uint32_t col = static_cast<uint32_t>(at);
  const int64_t left = static_cast<int64_t>(p.cols) - col;
  float dg[VE], db[VE];
#pragma unroll
  for (int i = 0; i < VE; ++i) dg[i] = 0.0f, db[i] = 0.0f;
#pragma unroll 4
  for (uint32_t row = blockIdx.y; row < p.rows; row += gridDim.y) {
    const typename X::Held h = X::load(p, row, col, left);
    const Raw<TX, VE> d = load_some<TX, VE>(
        static_cast<const TX*>(p.dy) + static_cast<int64_t>(row) * p.ld_dy + col, left);
    const float mean = p.mean[row], rstd = p.rstd[row];
    float xv[VE];
    X::values(h, xv);
#pragma unroll
    for (int i = 0; i < VE; ++i) {
      const float dy = to_f32(d.v[i]);
      dg[i] = fmaf(dy, (xv[i] - mean) * rstd, dg[i]);
      db[i] += dy;
    }
  }
  float* mine = p.partials + static_cast<uint64_t>(blockIdx.y) * 2u * p.cols;
#pragma unroll
  for (int i = 0; i < VE; ++i)
    if (i < left) {
      mine[col + i] = dg[i];
      mine[p.cols + col + i] = db[i];
    }
}

// dgamma and dbeta from ``parts`` rows of partial sums (none: zeros).  A block takes 32 columns of
// one of the two; warp w adds rows w, w + 8, ..., then the eight warps' sums are added in order.
template <typename TP>
__global__ void __launch_bounds__(256)
    norm_bwd_join_kernel(const float* __restrict__ partials, uint32_t parts, uint32_t cols,
                         TP* __restrict__ dgamma, TP* __restrict__ dbeta) {
  __shared__ float sums[8][32];
  grid_dependency_wait();
  grid_launch_dependents();
  const uint32_t lane = threadIdx.x & 31u, warp = threadIdx.x >> 5;
  const uint32_t col = blockIdx.x * 32u + lane;
  TP* out = blockIdx.y ? dbeta : dgamma;
  if (out == nullptr) return;
  float a = 0.0f;
  if (col < cols) {
    const float* src = partials + static_cast<uint64_t>(blockIdx.y) * cols + col;
#pragma unroll 8
    for (uint32_t i = warp; i < parts; i += 8u) a += src[static_cast<uint64_t>(i) * 2u * cols];
  }
  sums[warp][lane] = a;
  __syncthreads();
  if (warp == 0 && col < cols) {
#pragma unroll
    for (int w = 1; w < 8; ++w) a += sums[w][lane];
    out[col] = from_f32<TP>(a);
  }
}

}  // namespace tg
