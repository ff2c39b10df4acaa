// tg_norm_kernel.cuh -- layer norm over the rows of x [rows, cols], forward and backward.
//
// Forward, in 32 bits:  mean = sum x / cols,  rstd = 1 / sqrt(sum (x - mean)^2 / cols + eps),
// y = (x - mean) rstd gamma + beta, rounded once; optionally the 8-bit checkpoint of the rounded y
// as well (tg_rows.cuh), so that it need not be read again to be packed.
// Backward, with xh = (x - mean) rstd and g = dy gamma:
//   dx = rstd (g - sum g / cols - xh sum (g xh) / cols),  dgamma = sum_rows dy xh,
//   dbeta = sum_rows dy;  x is the tensor, or its 8-bit checkpoint.
// Both are bound by memory: a row stays on the SM from its one read to the result's write.
//
// Rows go to groups of G threads (G a multiple of 32), 16 values a thread (or 32, below); a CTA, one
// per SM, holds as many groups as its threads allow.  In the forward pass a group takes two rows a
// turn: one barrier, and one chain of shuffles, serves both.  Each thread copies its own values of
// the rows ahead to shared memory (cp.async), so that 64 KiB are on their way to an SM at any time.
// Rows of any alignment are read and written in whole 16-byte granules (UNAL, tg_rows.cuh).  Rows
// that a warp holds are left to tg_norm_short_kernel.cuh.
//
// The variance: each thread takes the mean of its own values and their squares about that mean
// (n, m, M2; fp32: about the mean of its first four, corrected for the rest); lanes, and then warps,
// are joined about the mean c of the first of them,
//   A = sum [M2 + n (m - c)^2],  B = sum n (m - c);  mean = c + B / n,  M2 = A - B^2 / n,
// two sums that run side by side.  No difference of large sums is formed, so a large mean costs no
// digits: B^2 / n <= (1 - 1 / k) sum n (m - c)^2 for k equal parts, at most 5 bits for 32.
#pragma once

#include <type_traits>

#include "tg_rows.cuh"

namespace tg {

constexpr int kNormMaxGroups = 15;   // one named barrier each
constexpr int kNormValues = 16;      // of a thread
// Threads of a CTA: 512 with 128 registers hold the parameters, the row's values and (backward) the
// sums over rows.  Rows of more than 8192 values take 1024 threads of 64 registers: one row a turn,
// parameters read again for each row, and (backward, 16-bit values only: 32-bit ones would need more
// shared memory than there is) the row's values taken from shared memory twice, some sums spilled.
constexpr int kNormThreads = 512;
constexpr int kNormWideThreads = 1024;
// Forward, 16-bit values: 512 threads of 32 values halve the shuffles, joins and barriers a value;
// the parameters come from shared memory up to 8192 columns and are read again above.  Taken for
// rows of more than 2048 values from 96 Ki values an SM on, else the start costs more: 8192 x 8192
// 53 us against 56 with 16 values a thread, 4000 x 7000 31 against 33, 4096 x 16384 70 against 85
// (1024 threads), but 100 x 8192 10.9 against 8.8.  fp32 rows would have one row a turn: 4800 x 16384
// 156 against 134.  (A row's last bits so depend on the number of rows.)
constexpr int kFwdLongValues = 32;
constexpr int kFwdLongCols = 2048, kFwdParamCols = 8192;
constexpr int64_t kFwdLongWork = 96 * 1024;   // values an SM

// Forward: rows a turn
template <int THREADS>
constexpr int kFwdRows = THREADS == kNormThreads ? 2 : 1;

// Turns whose rows have a place in shared memory: 64 KiB in flight besides the present one.
template <typename T, int THREADS, int VALUES>
constexpr int kFwdSlots =
    65536 / (THREADS * kFwdRows<THREADS> * VALUES * static_cast<int>(sizeof(T))) + 1;
template <typename T, int THREADS>
constexpr int kBwdSlots = 65536 / (THREADS * 2 * kNormValues * static_cast<int>(sizeof(T))) + 1;

// shared memory of ``warps`` warps for rows
template <typename T, int THREADS, int VALUES>
constexpr uint32_t norm_fwd_smem(uint32_t warps) {
  return warps * kFwdSlots<T, THREADS, VALUES> * kFwdRows<THREADS> * (VALUES / kVec<T>)*kStripBytes;
}
template <typename T, int THREADS>
constexpr uint32_t norm_bwd_smem(uint32_t warps) {
  return warps * 2 * kBwdSlots<T, THREADS> * (kNormValues / kVec<T>)*kStripBytes;
}

// How the rows lie.  kWholeRows: in whole 16-byte granules.  kAnyRows: anyhow; vectors are shifted
// out of two granules when they are read, and shifted back when they are written (tg_rows.cuh).
// kOneLead: anyhow, but in all the tensors alike, so that row r starts ``lead`` bytes into a granule
// in each; the rows of a CTA are a multiple of 8 apart and have one lead.  Backward, a thread takes
// granules instead of vectors: its columns begin lead values earlier, nothing is shifted, and only a
// row's first and last granule hold values that are not the row's.  (The sums' order, and with it the
// last bits of dx, then depends on the lead.)  Forward, the statistics are taken over vectors as ever,
// so that a row gives the same bits wherever it lies, and only y is written in granules; not with a
// checkpoint, whose blocks lie otherwise.
// Against kAnyRows, caches cold: forward 8000 x 4099 bf16 51 us instead of 87, 2000 x 4099 fp32 26
// instead of 36; backward 77 instead of 111, and 34 instead of 48; few rows alike.
enum Rows : int { kWholeRows, kOneLead, kAnyRows };

struct NormFwdParams {
  RowsOf x, y;
  const void* gamma;   // may be null (ones)
  const void* beta;    // may be null (zeros)
  uint32_t wide_params;     // both can be read in 16-byte vectors
  uint32_t shared_params;   // byte offset of their fp32 copies in shared memory; 0: none
  float* mean;         // may be null
  float* rstd;         // may be null
  uint8_t* q;          // checkpoint of y (KEEP)
  uint8_t* s;
  uint32_t rows, cols, blocks;
  float eps;
};

// The group's own barrier (id 0 is the CTA's); a group of one warp needs none.
__device__ __forceinline__ void group_sync(uint32_t group, uint32_t g_threads) {
  if (g_threads > 32u) asm volatile("bar.sync %0, %1;" ::"r"(group + 1u), "r"(g_threads) : "memory");
}

// How many of a row's values a warp of a group holds: strips w, w + g_warps, ... of 32 N values.
template <int N, int VALUES>
__device__ __forceinline__ float warp_share(uint32_t w, uint32_t g_warps, uint32_t cols) {
  uint32_t n = 0;
  for (uint32_t k = 0; k < VALUES / N; ++k) {
    const uint64_t at = static_cast<uint64_t>(k * g_warps + w) * (32u * N);
    if (at < cols) n += cols - at < 32u * N ? static_cast<uint32_t>(cols - at) : 32u * N;
  }
  return static_cast<float>(n);
}

template <typename TP, int N>
__device__ __forceinline__ void params_or(const void* p, uint32_t col, uint32_t cols, bool wide,
                                          float none, float (&v)[N]) {
  if (p) {
    load_params<TP, N>(static_cast<const TP*>(p), col, cols, wide, v);
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = none;
  }
}

// kOneLead: parameters of columns col + i, skip <= i < left (others: zero).
template <typename TP, int N>
__device__ __forceinline__ void params_between(const void* p, int col, int skip, int left, float none,
                                               float (&v)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i)
    v[i] = !p ? none : i >= skip && i < left ? to_f32(static_cast<const TP*>(p)[col + i]) : 0.0f;
}

// kOneLead: starts the copy of the lane's granule at p to shared memory.  ``inner``: all of it is
// the row's.
template <typename T>
__device__ __forceinline__ void stage_granule(uint32_t dst, const RowsOf& m, const char* p, int left,
                                              bool inner) {
  if (inner || (left > 0 && p >= m.base && p + 16 <= m.end)) {
    cp_async<16>(dst, p);
  } else if (left > 0) {   // at the matrix's ends
    const V16 r = load_granule<T>(p, m.base, m.end);
    st_shared_v4(dst, r.w[0], r.w[1], r.w[2], r.w[3]);
  }
}

// kOneLead: stores values skip to left - 1 of the granule at p.
template <typename T>
__device__ __forceinline__ void store_between(char* p, const V16& r, int skip, int left, bool inner) {
  if (inner) {
    store16(p, r);
  } else {
#pragma unroll
    for (int i = 0; i < kVec<T>; ++i)
      if (i >= skip && i < left) store_one<T>(p, r, i);
  }
}

// 1 / sqrt(a): rsqrtf is within 2 ulp, and one Newton step, r + r (1 - a r^2) / 2, takes that to
// about half of one.  Every value of a row is multiplied by it, so its error would move results to
// the other side of a rounding, a whole step of 1/16 in an 8-bit checkpoint.  0 gives infinity,
// infinity 0.
__device__ __forceinline__ float inverse_root(float a) {
  const float r = rsqrtf(a);
  const float e = fmaf(-a * r, r, 1.0f);
  return a > 0.0f && a < INFINITY ? fmaf(0.5f * r, e, r) : r;
}

// Adds ``rest``, the mean of the deviations from ``mean``, to it, and makes ``square``, the mean square
// about it, that about the new one.  Equal values so give their value, whatever the first sum lost.
// Only where the mean outweighs the deviations: they are rounded as the values are, all alike where
// the values have one exponent, which is more than a small mean's own sum loses.
__device__ __forceinline__ bool mean_outweighs(float mean, float square) {
  return square < mean * mean;
}
__device__ __forceinline__ void correct_mean(float& mean, float& square, float rest) {
  mean += rest;
  square = fmaxf(fmaf(-rest, rest, square), 0.0f);   // may round below zero
}

// Zeroes a warp's strips: those past a row's end stay so, and the values there count for nothing.
__device__ __forceinline__ void clear_strips(uint32_t at, uint32_t strips) {
  for (uint32_t o = (threadIdx.x & 31u) * 16u; o < strips * kStripBytes; o += 512u)
    st_shared_v4(at + o, 0u, 0u, 0u, 0u);
  __syncwarp();
}

// y of the lane's N values at column ``col`` (and their checkpoint), of which ``left`` are in the
// row; every lane of the warp calls it.
template <typename TX, bool UNAL, bool KEEP>
__device__ __forceinline__ void norm_write(const NormFwdParams& p, uint64_t row, uint32_t col,
                                           int left, const float (&v)[kVec<TX>], float mean,
                                           float rstd, const float (&g)[kVec<TX>],
                                           const float (&b)[kVec<TX>]) {
  constexpr int N = kVec<TX>;
  float o[N];
#pragma unroll
  for (int i = 0; i < N; ++i) o[i] = fmaf((v[i] - mean) * rstd, g[i], b[i]);
  const V16 out = rounded<TX>(o);
  store_vector<TX, UNAL>(p.y.base + static_cast<int64_t>(row) * p.y.pitch,
                         static_cast<int64_t>(col) * static_cast<int>(sizeof(TX)), out, left);
  if constexpr (KEEP) {
    values<TX>(out, o);   // as rounded
    if (left < N) {
#pragma unroll
      for (int i = 0; i < N; ++i) o[i] = i < left ? o[i] : 0.0f;
    }
    uint32_t q[N / 4];
    const uint32_t s = ckpt8_quantise<N>(o, q);
    const uint32_t b32 = col / kCkptBlock;
    if (b32 < p.blocks) {
      const uint64_t block = row * p.blocks + b32;
      store_kept<N>(p.q + block * kCkptBlock + col % kCkptBlock, q);
      if (col % kCkptBlock == 0) p.s[block] = static_cast<uint8_t>(s);
    }
  }
}

// Row r belongs to CTA r % gridDim.x, and its turns there to the groups in turn.
template <typename TX, typename TP, int ROWS, bool KEEP, int THREADS, int VALUES>
__global__ void __launch_bounds__(THREADS, 1)
    norm_fwd_kernel(const NormFwdParams p, const uint32_t g_threads) {
  extern __shared__ uint8_t staged[];
  constexpr int N = kVec<TX>, kItems = VALUES / N, R = kFwdRows<THREADS>;
  constexpr bool LEAD = ROWS == kOneLead, UNAL = ROWS == kAnyRows || LEAD;
  constexpr uint32_t kSlots = kFwdSlots<TX, THREADS, VALUES>;
  // parameters in registers, or in shared memory, or read again for each row
  constexpr bool kHeld = THREADS == kNormThreads && VALUES == kNormValues;
  constexpr bool kShared = VALUES == kFwdLongValues;
  static_assert(!LEAD || (THREADS == kNormThreads && !KEEP));
  constexpr bool kExact = sizeof(TX) == 4;   // sums that fp32 would round: below
  __shared__ float part[2][R][3][32];               // c, A and B of each warp
  const uint32_t lane = threadIdx.x & 31u, warp = threadIdx.x >> 5;
  const uint32_t groups = blockDim.x / g_threads, group = threadIdx.x / g_threads;
  const uint32_t g_warps = g_threads >> 5, wg = warp - group * g_warps;
  const int64_t row_bytes = static_cast<int64_t>(p.cols) * static_cast<int>(sizeof(TX));
  const uint32_t mine = smem_u32(staged) + warp * (kSlots * R * kItems * kStripBytes);
  // The statistics are always taken over vectors from the row's start, shifted out of their granules,
  // so that a row's have the same bits wherever it lies.
  uint32_t col[kItems];
  int left[kItems], n_mine = 0;
  bool inner[kItems];
#pragma unroll
  for (int k = 0; k < kItems; ++k) {
    const uint32_t v = (k * g_warps + wg) * 32u + lane;
    col[k] = v * N;
    left[k] = values_left<N>(v, p.cols);
    inner[k] = inner_vector<UNAL>(v * 16u, row_bytes);
    n_mine += left[k] > 0 ? left[k] : 0;
  }
  // kOneLead: y is written in granules, the thread's k-th of which holds columns col[k] - lead_n on
  const uint32_t lead =
      UNAL ? lead_of(p.x.base + static_cast<int64_t>(blockIdx.x) * p.x.pitch) : 0u;
  const int lead_n = static_cast<int>(lead / sizeof(TX));
  const int skip_0 = wg == 0u && lane == 0u ? lead_n : 0;
  auto skip = [=](int k) { return k == 0 ? skip_0 : 0; };   // values before the row's first
  auto end = [&](int k) { return values_left<N>(col[k] / N, p.cols + lead_n); };
  // values of this thread, of warp ``lane`` of the group, and of the row
  const float n_t = static_cast<float>(n_mine);
  const float n_l = lane < g_warps ? warp_share<N, VALUES>(lane, g_warps, p.cols) : 0.0f;
  const float inv_l = n_l > 0.0f ? 1.0f / n_l : 0.0f;
  const float inv_row = 1.0f / static_cast<float>(p.cols);
  grid_dependency_wait();
  grid_launch_dependents();

  float g[kHeld ? kItems : 1][N], b[kHeld ? kItems : 1][N];
  if constexpr (kHeld) {
#pragma unroll
    for (int k = 0; k < kItems; ++k) {
      if constexpr (LEAD) {
        const int at = static_cast<int>(col[k]) - lead_n;
        params_between<TP, N>(p.gamma, at, skip(k), end(k), 1.0f, g[k]);
        params_between<TP, N>(p.beta, at, skip(k), end(k), 0.0f, b[k]);
      } else {
        params_or<TP, N>(p.gamma, col[k], p.cols, p.wide_params, 1.0f, g[k]);
        params_or<TP, N>(p.beta, col[k], p.cols, p.wide_params, 0.0f, b[k]);
      }
    }
  }
  // fp32 copies for every vector of the row, four columns of each of 32 lanes' vectors after
  // the other, so that a warp reads them without meeting in a bank: gamma, then beta
  const uint32_t shared_g = smem_u32(staged) + p.shared_params;
  const uint32_t shared_b = shared_g + g_threads * VALUES * 4u;
  if (kShared && p.shared_params) {
    for (uint32_t v = threadIdx.x; v < kItems * g_threads; v += blockDim.x) {
      float t[2][N];
      if constexpr (LEAD) {
        const int at = static_cast<int>(v * N) - lead_n, n = values_left<N>(v, p.cols + lead_n);
        params_between<TP, N>(p.gamma, at, v == 0u ? lead_n : 0, n, 1.0f, t[0]);
        params_between<TP, N>(p.beta, at, v == 0u ? lead_n : 0, n, 0.0f, t[1]);
      } else {
        params_or<TP, N>(p.gamma, v * N, p.cols, p.wide_params, 1.0f, t[0]);
        params_or<TP, N>(p.beta, v * N, p.cols, p.wide_params, 0.0f, t[1]);
      }
#pragma unroll
      for (int j = 0; j < N / 4; ++j) {
        const uint32_t at = ((v / 32u * (N / 4) + j) * 32u + v % 32u) * 16u;
#pragma unroll
        for (int h = 0; h < 2; ++h)
          st_shared_v4((h ? shared_b : shared_g) + at, __float_as_uint(t[h][4 * j]),
                       __float_as_uint(t[h][4 * j + 1]), __float_as_uint(t[h][4 * j + 2]),
                       __float_as_uint(t[h][4 * j + 3]));
      }
    }
    __syncthreads();
  }
  auto params_of = [&](int k, float (&gg)[N], float (&bb)[N]) {   // not held
    if (kShared && p.shared_params) {
#pragma unroll
      for (int j = 0; j < N / 4; ++j) {
        const uint32_t at = (((k * g_warps + wg) * (N / 4) + j) * 32u + lane) * 16u;
        const V16 x = ld_shared_v16(shared_g + at), y = ld_shared_v16(shared_b + at);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          gg[4 * j + i] = __uint_as_float(x.w[i]);
          bb[4 * j + i] = __uint_as_float(y.w[i]);
        }
      }
    } else {
      params_or<TP, N>(p.gamma, col[k], p.cols, p.wide_params, 1.0f, gg);
      params_or<TP, N>(p.beta, col[k], p.cols, p.wide_params, 0.0f, bb);
    }
  };
  const uint64_t step = static_cast<uint64_t>(gridDim.x) * groups;
  auto stage = [&](uint64_t row, uint32_t slot) {   // rows row and row + step
#pragma unroll
    for (int r = 0; r < R; ++r) {
      if (row + r * step < p.rows) {
        const char* at = p.x.base + static_cast<int64_t>(row + r * step) * p.x.pitch;
#pragma unroll
        for (int k = 0; k < kItems; ++k)
          stage_vector<TX, UNAL>(mine + ((slot * R + r) * kItems + k) * kStripBytes, p.x, at,
                                 col[k] * static_cast<uint32_t>(sizeof(TX)), row_bytes, inner[k]);
      }
    }
    cp_async_commit();
  };
  uint64_t row = blockIdx.x + static_cast<uint64_t>(gridDim.x) * group, ahead = row;
  uint32_t slot = 0;
  clear_strips(mine, kSlots * R * kItems);
#pragma unroll
  for (uint32_t i = 0; i + 1 < kSlots; ++i, ahead += R * step) stage(ahead, i);
  for (uint32_t turn = 0; row < p.rows; row += R * step, ++turn) {
    stage(ahead, slot == 0u ? kSlots - 1u : slot - 1u);
    ahead += R * step;
    cp_async_wait<kSlots - 1>();
    __syncwarp();
    // a row past the end: what the slot holds, reduced and not written
    float v[R][kItems][N], c[R], ab[2 * R];   // ab: A and B of each row
#pragma unroll
    for (int r = 0; r < R; ++r) {
      float s = 0.0f;
#pragma unroll
      for (int k = 0; k < kItems; ++k) {
        values<TX>(staged_vector<TX, UNAL>(mine + ((slot * R + r) * kItems + k) * kStripBytes, lead),
                   v[r][k]);
        if (UNAL && left[k] < N && (!kExact || k == 0)) {
#pragma unroll
          for (int i = 0; i < N; ++i) v[r][k][i] = i < left[k] ? v[r][k][i] : kExact ? v[r][0][0] : 0.0f;
        }
        if constexpr (!kExact) {
#pragma unroll
          for (int i = 0; i < N; ++i) s += v[r][k][i];
        }
      }
      // Where all values are one, so is their mean.  32 values of 16 bits add up exactly; of fp32 ones,
      // which do not, four do, in pairs: squares are taken about the first vector's mean, and ``low`` is
      // what the thread's mean has beyond it.
      auto over_n = [&](float a) { return n_mine == VALUES ? a * (1.0f / VALUES) : a / n_t; };
      float m, m2 = 0.0f, off = 0.0f, low = 0.0f;
      if constexpr (kExact)
        m = 0.25f * ((v[r][0][0] + v[r][0][1]) + (v[r][0][2] + v[r][0][3]));
      else
        m = n_mine > 0 ? over_n(s) : 0.0f;
#pragma unroll
      for (int k = 0; k < kItems; ++k) {
        float q = 0.0f, e = 0.0f;
        if (UNAL && left[k] < N) {   // what is not the row's deviates by nothing
#pragma unroll
          for (int i = 0; i < N; ++i) v[r][k][i] = i < left[k] ? v[r][k][i] : m;
        }
#pragma unroll
        for (int i = 0; i < N; ++i) {
          const float d = v[r][k][i] - m;
          q = fmaf(d, d, q);
          if constexpr (kExact) e += d;
        }
        m2 += left[k] > 0 ? q : 0.0f;
        if constexpr (kExact) off += left[k] > 0 ? e : 0.0f;
      }
      if (kExact && n_mine > 0) {
        low = over_n(off);
        m2 = fmaf(-off, low, m2);
      }
      // lane 0 holds values wherever its warp holds any
      c[r] = __shfl_sync(0xffffffffu, kExact ? m + low : m, 0);
      const float d = n_mine > 0 ? (kExact ? (m - c[r]) + low : m - c[r]) : 0.0f;
      ab[2 * r + 1] = n_t * d;
      ab[2 * r] = fmaf(ab[2 * r + 1], d, m2);
    }
    float sums = warp_sums(ab);
    if (g_warps > 1u) {
      if (lane % (16 / R) == 0u) part[turn & 1u][lane / (32 / R)][1 + lane / (16 / R) % 2][warp] = sums;
      if (lane == 0u) {
#pragma unroll
        for (int r = 0; r < R; ++r) part[turn & 1u][r][0][warp] = c[r];
      }
      group_sync(group, g_threads);
      const uint32_t w = warp - wg + (lane < g_warps ? lane : 0u);
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const float bw = part[turn & 1u][r][2][w], dw = bw * inv_l;
        const float cw = part[turn & 1u][r][0][w], mw = cw + dw;
        const float m2 = fmaf(-bw, dw, part[turn & 1u][r][1][w]);
        c[r] = __shfl_sync(0xffffffffu, mw, 0);
        const float d = n_l > 0.0f ? (kExact ? (cw - c[r]) + dw : mw - c[r]) : 0.0f;
        ab[2 * r + 1] = n_l * d;
        ab[2 * r] = n_l > 0.0f ? fmaf(ab[2 * r + 1], d, m2) : 0.0f;
      }
      sums = warp_sums(ab);
    }
    float mean[R], rstd[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const float sa = sum_of<2 * R>(sums, 2 * r), sb = sum_of<2 * R>(sums, 2 * r + 1);
      const float d = sb * inv_row;
      mean[r] = c[r] + d;
      const float m2 = fmaf(-sb, d, sa);   // may round below zero
      rstd[r] = inverse_root((m2 < 0.0f ? 0.0f : m2) * inv_row + p.eps);
    }
    if (wg == 0u && lane == 0u) {
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const uint64_t at = row + r * step;
        if (at >= p.rows) break;
        if (p.mean) p.mean[at] = mean[r];
        if (p.rstd) p.rstd[at] = rstd[r];
      }
    }
    __syncwarp();
#pragma unroll
    for (int k = 0; k < kItems; ++k) {
      if constexpr (!kHeld) params_of(k, g[0], b[0]);
#pragma unroll
      for (int r = 0; r < R; ++r) {
        if (row + r * step >= p.rows) break;
        if constexpr (LEAD) {
          float o[N];
          values<TX>(ld_shared_v16(mine + ((slot * R + r) * kItems + k) * kStripBytes + lane * 16u),
                     o);
#pragma unroll
          for (int i = 0; i < N; ++i) o[i] = fmaf((o[i] - mean[r]) * rstd[r], g[kHeld ? k : 0][i], b[kHeld ? k : 0][i]);
          const int n = end(k);
          store_between<TX>(p.y.base + static_cast<int64_t>(row + r * step) * p.y.pitch - lead +
                                col[k] * static_cast<uint32_t>(sizeof(TX)),
                            rounded<TX>(o), skip(k), n, n == N && skip(k) == 0);
        } else {
          norm_write<TX, UNAL, KEEP>(p, row + r * step, col[k], left[k], v[r][k], mean[r], rstd[r],
                                     g[kHeld ? k : 0], b[kHeld ? k : 0]);
        }
      }
    }
    __syncwarp();   // every lane has read the slot before it is filled again
    slot = slot + 1u == kSlots ? 0u : slot + 1u;
  }
  cp_async_wait<0>();
}

// Any width: the CTA walks its row three times (mean; squares about it, and what the mean lacks; y);
// the second and third reads come from the L2.
template <typename TX, typename TP, bool UNAL, bool KEEP>
__global__ void __launch_bounds__(1024) norm_fwd_long_kernel(const NormFwdParams p) {
  __shared__ float part[2][2][32];
  constexpr int N = kVec<TX>;
  const uint32_t lane = threadIdx.x & 31u, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  grid_dependency_wait();
  grid_launch_dependents();
  const uint32_t row = blockIdx.x;
  const char* x = p.x.base + static_cast<int64_t>(row) * p.x.pitch;
  const int64_t row_bytes = static_cast<int64_t>(p.cols) * static_cast<int>(sizeof(TX));
  const uint32_t end = ((p.cols + N - 1) / N + 31u) & ~31u;   // vectors, whole strips
  float mean = 0.0f;
  auto walk = [&](auto which, float& sum, float& squares) {   // of deviations from ``mean``
    constexpr int pass = decltype(which)::value;
    float a = 0.0f, q = 0.0f;
    for (uint32_t j = threadIdx.x; j < end; j += blockDim.x) {
      const int64_t left = static_cast<int64_t>(p.cols) - static_cast<int64_t>(j) * N;
      float v[N];
      values<TX>(load_vector<TX, UNAL>(p.x, x, static_cast<int64_t>(j) * 16, row_bytes), v);
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const float d = i < left ? v[i] - mean : 0.0f;
        a += d;
        if constexpr (pass) q = fmaf(d, d, q);
      }
    }
    a = warp_sum(a);
    if constexpr (pass) q = warp_sum(q);
    if (lane == 0) {
      part[pass][0][warp] = a;
      part[pass][1][warp] = q;
    }
    __syncthreads();
    sum = warp_sum(lane < warps ? part[pass][0][lane] : 0.0f) / static_cast<float>(p.cols);
    squares = warp_sum(lane < warps ? part[pass][1][lane] : 0.0f) / static_cast<float>(p.cols);
  };
  float first, rest, square;
  walk(std::integral_constant<int, 0>(), first, square);
  mean = first;
  walk(std::integral_constant<int, 1>(), rest, square);
  if (mean_outweighs(mean, square)) correct_mean(mean, square, rest);
  const float rstd = inverse_root(square + p.eps);
  if (threadIdx.x == 0) {
    if (p.mean) p.mean[row] = mean;
    if (p.rstd) p.rstd[row] = rstd;
  }
  for (uint32_t j = threadIdx.x; j < end; j += blockDim.x) {
    float v[N];
    values<TX>(load_vector<TX, UNAL>(p.x, x, static_cast<int64_t>(j) * 16, row_bytes), v);
    float g[N], b[N];
    params_or<TP, N>(p.gamma, j * N, p.cols, p.wide_params, 1.0f, g);
    params_or<TP, N>(p.beta, j * N, p.cols, p.wide_params, 0.0f, b);
    norm_write<TX, UNAL, KEEP>(p, row, j * N, values_left<N>(j, p.cols), v, mean, rstd, g, b);
  }
}

// ---------------------------------------------------------------- backward
struct NormBwdParams {
  RowsOf dy, dx;
  RowsOf x;              // the tensor (not KEPT)
  const uint8_t* q;      // the checkpoint of x (KEPT)
  const uint8_t* s;
  const void* gamma;     // may be null (ones)
  uint32_t wide_params;
  const float* mean;
  const float* rstd;
  float* partials;       // [parts][2][part_cols] sums of dy xh and of dy; null: not wanted
  uint32_t part_cols;    // a multiple of 32, at least cols (kOneLead: and the largest lead)
  uint32_t rows, cols, blocks;
};

// The lane's N values of x at vector ``v`` of the row, straight from memory (every lane calls it).
template <typename TX, bool UNAL, bool KEPT>
__device__ __forceinline__ void x_values(const NormBwdParams& p, uint32_t row, uint32_t v,
                                         int64_t row_bytes, float (&out)[kVec<TX>]) {
  constexpr int N = kVec<TX>;
  if constexpr (KEPT) {
    uint32_t q[N / 4] = {}, s = 127u;
    const uint64_t col = static_cast<uint64_t>(v) * N;
    if (col < p.cols) {
      const uint64_t b = static_cast<uint64_t>(row) * p.blocks + col / kCkptBlock;
      load_kept<N>(p.q + b * kCkptBlock + col % kCkptBlock, q);
      s = p.s[b];
    }
    kept_values<N>(q, s, out);
  } else {
    const char* at = p.x.base + static_cast<int64_t>(row) * p.x.pitch;
    values<TX>(load_vector<TX, UNAL>(p.x, at, static_cast<int64_t>(v) * 16, row_bytes), out);
  }
}

// As the forward kernel; each thread keeps the sums of dy xh and dy of its own columns in registers
// over all its rows.  At the end the groups of a CTA add up in order, the CTA writes one row of
// partial sums, and norm_bwd_join_kernel adds those in a fixed order, so the result does not depend
// on timing.  A staged strip of a checkpoint holds N bytes a lane; scales, like the statistics, are
// read into registers a row ahead.
template <typename TX, typename TP, int ROWS, bool KEPT, int THREADS>
__global__ void __launch_bounds__(THREADS, 1)
    norm_bwd_kernel(const NormBwdParams p, const uint32_t g_threads) {
  extern __shared__ uint8_t staged[];
  constexpr int N = kVec<TX>, kItems = kNormValues / N;
  constexpr uint32_t kSlots = kBwdSlots<TX, THREADS>;
  constexpr bool UNAL = ROWS == kAnyRows, LEAD = ROWS == kOneLead;
  constexpr bool kHeld = THREADS == kNormThreads;   // gamma and the row's values in registers
  __shared__ float part[2][2][32];
  const uint32_t lane = threadIdx.x & 31u, warp = threadIdx.x >> 5;
  const uint32_t groups = blockDim.x / g_threads, group = threadIdx.x / g_threads;
  const uint32_t g_warps = g_threads >> 5, wg = warp - group * g_warps;
  const int64_t row_bytes = static_cast<int64_t>(p.cols) * static_cast<int>(sizeof(TX));
  // per warp and slot: kItems strips of dy, then of x
  const uint32_t mine = smem_u32(staged) + warp * (kSlots * 2 * kItems * kStripBytes);
  const float inv_cols = 1.0f / static_cast<float>(p.cols);
  static_assert(!LEAD || (kHeld && !KEPT));
  const uint32_t lead =   // kOneLead: bytes, and values
      LEAD ? lead_of(p.dy.base + static_cast<int64_t>(blockIdx.x) * p.dy.pitch) : 0u;
  const int lead_n = static_cast<int>(lead / sizeof(TX));
  uint32_t col[kItems];   // kOneLead: counted from the row's first granule
  int left[kItems];
  bool inner[kItems];
  const int skip_0 = wg == 0u && lane == 0u ? lead_n : 0;
  auto skip = [=](int k) { return k == 0 ? skip_0 : 0; };   // values before the row's first
#pragma unroll
  for (int k = 0; k < kItems; ++k) {
    const uint32_t v = (k * g_warps + wg) * 32u + lane;
    col[k] = v * N;
    left[k] = values_left<N>(v, p.cols + lead_n);
    inner[k] = LEAD ? left[k] == N && skip(k) == 0 : inner_vector<UNAL>(v * 16u, row_bytes);
  }
  grid_dependency_wait();
  grid_launch_dependents();

  float held_g[kHeld ? kItems : 1][N];
  if constexpr (kHeld) {
#pragma unroll
    for (int k = 0; k < kItems; ++k) {
      if constexpr (LEAD)
        params_between<TP, N>(p.gamma, static_cast<int>(col[k]) - lead_n, skip(k), left[k], 1.0f,
                              held_g[k]);
      else
        params_or<TP, N>(p.gamma, col[k], p.cols, p.wide_params, 1.0f, held_g[k]);
    }
  }
  auto gamma_at = [&](int k, float (&g)[N]) {
    if constexpr (kHeld) {
#pragma unroll
      for (int i = 0; i < N; ++i) g[i] = held_g[k][i];
    } else {
      params_or<TP, N>(p.gamma, col[k], p.cols, p.wide_params, 1.0f, g);
    }
  };
  const uint64_t step = static_cast<uint64_t>(gridDim.x) * groups;
  auto stage = [&](uint64_t row, uint32_t slot) {
    const uint32_t at = mine + slot * (2 * kItems * kStripBytes);
    if (row < p.rows) {
      const char* dy = p.dy.base + static_cast<int64_t>(row) * p.dy.pitch;
#pragma unroll
      for (int k = 0; k < kItems; ++k) {
        const uint32_t byte = col[k] * static_cast<uint32_t>(sizeof(TX));
        if constexpr (LEAD)
          stage_granule<TX>(at + k * kStripBytes + lane * 16u, p.dy, dy - lead + byte, left[k],
                            inner[k]);
        else
          stage_vector<TX, UNAL>(at + k * kStripBytes, p.dy, dy, byte, row_bytes, inner[k]);
        const uint32_t xs = at + (kItems + k) * kStripBytes;
        if constexpr (KEPT) {
          if (left[k] > 0)
            cp_async<N>(xs + lane * N, p.q + row * p.blocks * kCkptBlock + col[k]);
        } else {
          const char* x = p.x.base + static_cast<int64_t>(row) * p.x.pitch;
          if constexpr (LEAD)
            stage_granule<TX>(xs + lane * 16u, p.x, x - lead + byte, left[k], inner[k]);
          else
            stage_vector<TX, UNAL>(xs, p.x, x, byte, row_bytes, inner[k]);
        }
      }
    }
    cp_async_commit();
  };
  uint32_t scale[kItems] = {};
  auto scales_of = [&](uint64_t row, uint32_t (&to)[kItems]) {
#pragma unroll
    for (int k = 0; k < kItems; ++k)
      to[k] = KEPT && left[k] > 0 ? p.s[row * p.blocks + col[k] / kCkptBlock] : 127u;
  };
  // the lane's dy and xh of its k-th vector, from the row's slot; past the row's end both are
  // zero (!kHeld and kWholeRows: dy alone)
  auto values_at = [&](uint64_t row, uint32_t slot, int k, float mean, float rstd, float (&dy)[N],
                       float (&xh)[N]) {
    const uint32_t at = mine + slot * (2 * kItems * kStripBytes);
    const uint32_t lead_dy =
        UNAL ? lead_of(p.dy.base + static_cast<int64_t>(row) * p.dy.pitch) : 0u;
    values<TX>(staged_vector<TX, UNAL>(at + k * kStripBytes, lead_dy), dy);
    const uint32_t xs = at + (kItems + k) * kStripBytes;
    // A lane past the row's end has zeros in its strips.  kWholeRows: it takes them about zero, since
    // mean * rstd may be infinite and zero times that would not be zero (!kHeld: it skips its sums).
    const float about = !kHeld || ROWS != kWholeRows || left[k] > 0 ? mean : 0.0f;
    if constexpr (KEPT) {
      uint32_t q[N / 4];
      if constexpr (N == 8)
        asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(q[0]), "=r"(q[1]) : "r"(xs + lane * 8u) : "memory");
      else
        q[0] = ld_shared_u32(xs + lane * 4u);
      kept_less<N>(q, scale[k], about, xh);
#pragma unroll
      for (int i = 0; i < N; ++i) xh[i] *= rstd;
    } else {
      const uint32_t lead_x = UNAL ? lead_of(p.x.base + static_cast<int64_t>(row) * p.x.pitch) : 0u;
      values<TX>(staged_vector<TX, UNAL>(xs, lead_x), xh);
#pragma unroll
      for (int i = 0; i < N; ++i) xh[i] = (xh[i] - about) * rstd;
    }
    if (UNAL || (LEAD && !inner[k])) {
#pragma unroll
      for (int i = 0; i < N; ++i) {
        dy[i] = i >= skip(k) && i < left[k] ? dy[i] : 0.0f;
        xh[i] = i >= skip(k) && i < left[k] ? xh[i] : 0.0f;
      }
    }
  };

  float dg[kItems][N], db[kItems][N];
#pragma unroll
  for (int k = 0; k < kItems; ++k)
#pragma unroll
    for (int i = 0; i < N; ++i) dg[k][i] = db[k][i] = 0.0f;
  uint64_t row = blockIdx.x + static_cast<uint64_t>(gridDim.x) * group, ahead = row;
  uint32_t slot = 0;
  float mean = 0.0f, rstd = 0.0f;
  if (row < p.rows) {
    mean = p.mean[row];
    rstd = p.rstd[row];
    scales_of(row, scale);
  }
  clear_strips(mine, kSlots * 2 * kItems);
#pragma unroll
  for (uint32_t i = 0; i + 1 < kSlots; ++i, ahead += step) stage(ahead, i);
  for (uint32_t turn = 0; row < p.rows; row += step, ++turn) {
    stage(ahead, slot == 0u ? kSlots - 1u : slot - 1u);
    ahead += step;
    float next_mean = 0.0f, next_rstd = 0.0f;
    uint32_t next_scale[kItems] = {};
    if (row + step < p.rows) {
      next_mean = p.mean[row + step];
      next_rstd = p.rstd[row + step];
      scales_of(row + step, next_scale);
    }
    cp_async_wait<kSlots - 1>();
    __syncwarp();
    float s[2] = {0.0f, 0.0f};   // sums of dy gamma, and of it times xh
    float hold_g[kHeld ? kItems : 1][N], hold_x[kHeld ? kItems : 1][N];
#pragma unroll
    for (int k = 0; k < kItems; ++k) {
      if (!kHeld && ROWS == kWholeRows && left[k] <= 0) continue;
      float dy[N], xh[N], g[N];
      gamma_at(k, g);
      values_at(row, slot, k, mean, rstd, dy, xh);
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const float gd = dy[i] * g[i];
        s[0] += gd;
        s[1] = fmaf(gd, xh[i], s[1]);
        dg[k][i] = fmaf(dy[i], xh[i], dg[k][i]);
        db[k][i] += dy[i];
        if constexpr (kHeld) {
          hold_g[k][i] = gd;
          hold_x[k][i] = xh[i];
        }
      }
    }
    float sums = warp_sums(s);
    if (g_warps > 1u) {
      if (lane % 16u == 0u) part[turn & 1u][lane / 16u][warp] = sums;
      group_sync(group, g_threads);
      s[0] = lane < g_warps ? part[turn & 1u][0][warp - wg + lane] : 0.0f;
      s[1] = lane < g_warps ? part[turn & 1u][1][warp - wg + lane] : 0.0f;
      sums = warp_sums(s);
    }
    // dx = rstd gd - rstd c1 - xh rstd c2
    const float c1 = sum_of<2>(sums, 0) * inv_cols * rstd;
    const float c2 = sum_of<2>(sums, 1) * inv_cols * rstd;
    char* out = p.dx.base + static_cast<int64_t>(row) * p.dx.pitch;
#pragma unroll
    for (int k = 0; k < kItems; ++k) {
      float dx[N];
      if constexpr (kHeld) {
#pragma unroll
        for (int i = 0; i < N; ++i)
          dx[i] = fmaf(-hold_x[k][i], c2, fmaf(hold_g[k][i], rstd, -c1));
      } else {   // the row again, from shared memory
        float xh[N], g[N];
        values_at(row, slot, k, mean, rstd, dx, xh);
        gamma_at(k, g);
#pragma unroll
        for (int i = 0; i < N; ++i) dx[i] = fmaf(-xh[i], c2, fmaf(dx[i] * g[i], rstd, -c1));
      }
      const int64_t byte = static_cast<int64_t>(col[k]) * static_cast<int>(sizeof(TX));
      if constexpr (LEAD)
        store_between<TX>(out - lead + byte, rounded<TX>(dx), skip(k), left[k], inner[k]);
      else
        store_vector<TX, UNAL>(out, byte, rounded<TX>(dx), left[k]);
    }
    __syncwarp();   // every lane has read the slot before it is filled again
    slot = slot + 1u == kSlots ? 0u : slot + 1u;
    mean = next_mean;
    rstd = next_rstd;
#pragma unroll
    for (int k = 0; k < kItems; ++k) scale[k] = next_scale[k];
  }
  cp_async_wait<0>();
  if (p.partials == nullptr) return;
  float* out = p.partials + static_cast<uint64_t>(blockIdx.x) * 2u * p.part_cols;
  float* sums = reinterpret_cast<float*>(staged);   // [2][part_cols], once staging is over
  // kOneLead: columns counted from the first granule here too; the join knows each CTA's lead
  if (groups > 1u) __syncthreads();
  for (uint32_t g = 0; g < groups; ++g) {           // the groups add up one by one
    if (group == g) {
#pragma unroll
      for (int k = 0; k < kItems; ++k) {
#pragma unroll
        for (int i = 0; i < N; i += 4) {
          const uint32_t col = ((k * g_warps + wg) * 32u + lane) * N + i;
          if (col >= p.part_cols) continue;
          float4 a = make_float4(dg[k][i], dg[k][i + 1], dg[k][i + 2], dg[k][i + 3]);
          float4 b = make_float4(db[k][i], db[k][i + 1], db[k][i + 2], db[k][i + 3]);
          float4* sa = reinterpret_cast<float4*>(sums + col);
          float4* sb = reinterpret_cast<float4*>(sums + p.part_cols + col);
          if (g > 0u) {
            const float4 c = *sa, d = *sb;
            a.x += c.x; a.y += c.y; a.z += c.z; a.w += c.w;
            b.x += d.x; b.y += d.y; b.z += d.z; b.w += d.w;
          }
          if (g + 1u == groups) {
            *reinterpret_cast<float4*>(out + col) = a;
            *reinterpret_cast<float4*>(out + p.part_cols + col) = b;
          } else {
            *sa = a;
            *sb = b;
          }
        }
      }
    }
    if (g + 1u < groups) __syncthreads();
  }
}

// Any width: a CTA walks its row twice (sums, then dx; the second read comes from the L2), and
// norm_bwd_cols_kernel reads x and dy once more for the sums over rows.
template <typename TX, typename TP, bool UNAL, bool KEPT>
__global__ void __launch_bounds__(1024) norm_bwd_long_kernel(const NormBwdParams p) {
  __shared__ float2 part[32];
  constexpr int N = kVec<TX>;
  const uint32_t lane = threadIdx.x & 31u, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  grid_dependency_wait();
  grid_launch_dependents();
  const uint32_t row = blockIdx.x;
  const float mean = p.mean[row], rstd = p.rstd[row];
  const int64_t row_bytes = static_cast<int64_t>(p.cols) * static_cast<int>(sizeof(TX));
  const char* dy_row = p.dy.base + static_cast<int64_t>(row) * p.dy.pitch;
  const uint32_t end = ((p.cols + N - 1) / N + 31u) & ~31u;   // vectors, whole strips
  float c1 = 0.0f, c2 = 0.0f;
#pragma unroll 1
  for (int pass = 0; pass < 2; ++pass) {
    for (uint32_t j = threadIdx.x; j < end; j += blockDim.x) {
      const int64_t left = static_cast<int64_t>(p.cols) - static_cast<int64_t>(j) * N;
      float x[N], dy[N], g[N];
      x_values<TX, UNAL, KEPT>(p, row, j, row_bytes, x);
      values<TX>(load_vector<TX, UNAL>(p.dy, dy_row, static_cast<int64_t>(j) * 16, row_bytes), dy);
#pragma unroll
      for (int i = 0; i < N; ++i) g[i] = 1.0f;
      if (p.gamma)
        load_params<TP, N>(static_cast<const TP*>(p.gamma), j * N, p.cols, p.wide_params, g);
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const float xh = i < left ? (x[i] - mean) * rstd : 0.0f;
        const float d = i < left ? dy[i] : 0.0f;
        if (pass == 0) {
          c1 = fmaf(d, g[i], c1);
          c2 = fmaf(d * g[i], xh, c2);
        }
        dy[i] = rstd * (fmaf(d, g[i], -c1) - xh * c2);
      }
      if (pass == 1)
        store_vector<TX, UNAL>(p.dx.base + static_cast<int64_t>(row) * p.dx.pitch,
                               static_cast<int64_t>(j) * 16, rounded<TX>(dy),
                               values_left<N>(j, p.cols));
    }
    if (pass == 0) {
      c1 = warp_sum(c1);
      c2 = warp_sum(c2);
      if (lane == 0) part[warp] = make_float2(c1, c2);
      __syncthreads();
      const float2 other = lane < warps ? part[lane] : make_float2(0.0f, 0.0f);
      c1 = warp_sum(other.x) / static_cast<float>(p.cols);
      c2 = warp_sum(other.y) / static_cast<float>(p.cols);
    }
  }
}

// Sums over rows for any width: thread t of block (i, j) takes N columns and rows j, j + parts, ...
template <typename TX, bool UNAL, bool KEPT>
__global__ void __launch_bounds__(128) norm_bwd_cols_kernel(const NormBwdParams p) {
  constexpr int N = kVec<TX>;
  grid_dependency_wait();
  grid_launch_dependents();
  const uint32_t v = blockIdx.x * blockDim.x + threadIdx.x;
  const int64_t row_bytes = static_cast<int64_t>(p.cols) * static_cast<int>(sizeof(TX));
  float dg[N], db[N];
#pragma unroll
  for (int i = 0; i < N; ++i) dg[i] = db[i] = 0.0f;
#pragma unroll 4
  for (uint32_t row = blockIdx.y; row < p.rows; row += gridDim.y) {
    float x[N], dy[N];
    x_values<TX, UNAL, KEPT>(p, row, v, row_bytes, x);
    values<TX>(load_vector<TX, UNAL>(p.dy, p.dy.base + static_cast<int64_t>(row) * p.dy.pitch,
                                     static_cast<int64_t>(v) * 16, row_bytes),
               dy);
    const float mean = p.mean[row], rstd = p.rstd[row];
#pragma unroll
    for (int i = 0; i < N; ++i) {
      dg[i] = fmaf(dy[i], (x[i] - mean) * rstd, dg[i]);
      db[i] += dy[i];
    }
  }
  float* out = p.partials + static_cast<uint64_t>(blockIdx.y) * 2u * p.part_cols;
#pragma unroll
  for (int i = 0; i < N; i += 4) {
    const uint64_t col = static_cast<uint64_t>(v) * N + i;
    if (col >= p.part_cols) continue;
    *reinterpret_cast<float4*>(out + col) = make_float4(dg[i], dg[i + 1], dg[i + 2], dg[i + 3]);
    *reinterpret_cast<float4*>(out + p.part_cols + col) =
        make_float4(db[i], db[i + 1], db[i + 2], db[i + 3]);
  }
}

// dgamma and dbeta from ``parts`` rows of partial sums (none: zeros).  A block takes 32 columns of
// one of the two; warp w adds rows w, w + 8, ..., then the eight warps' sums are added in order.
// Row i's columns begin (first + i * apart) % 16 / size values in (kOneLead; else first = apart = 0).
template <typename TP>
__global__ void __launch_bounds__(256)
    norm_bwd_join_kernel(const float* __restrict__ partials, uint32_t parts, uint32_t part_cols,
                         uint32_t cols, uint32_t first, uint32_t apart, uint32_t size_log2,
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
    // the same for a warp's rows, 8 apart
    const uint32_t lead = (first + warp * apart) % 16u >> size_log2;
    const float* src = partials + static_cast<uint64_t>(blockIdx.y) * part_cols + col + lead;
#pragma unroll 8
    for (uint32_t i = warp; i < parts; i += 8u) a += src[static_cast<uint64_t>(i) * 2u * part_cols];
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
