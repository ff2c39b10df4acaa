// tg_few_kernel.cuh -- the products of tg_linear_kernel.cuh for at most 64 rows: a token or a few that are
// being generated, a short text's loss.
//
//   D[r, n] = sum_k A[r, k] B[k, n]
//
// What bounds them is reading B, the weights, once: 2 bytes for at most 128 operations.  The pair
// kernel's MMA has 256 rows whatever there are, so it multiplies 250 rows of zeros as long as the weights
// take to arrive; and its tiles are few and large.  Here the weights are the MMA's M operand (128 of
// their rows or columns, cta_group::1) and the rows its N, padded to 16, 32 or 64: 32 cycles for each
// 16 of K where the weights' 4 KiB take about 90 to arrive.
//
// A CTA has one tile of 128 results per row.  Few tiles: a cluster of up to 8 CTAs shares one along K; each
// adds its range, then the sums are handed out by rows through distributed shared memory, every CTA
// adds its rows' in the order of the ranges and finishes them.  Nothing goes through global memory
// and no second launch follows.  Two CTAs an SM.  Where even clusters leave most SMs idle before a long
// K (a gradient towards x over a large vocabulary), K is cut between ``groups`` of clusters first, whose
// fp32 sums linear_join_kernel adds in order.
//
// Gradients that were rounded to 16 bits on the way come in two terms, what was rounded and what that
// left: with few rows their errors do not average out in a result (of one row, a gradient towards x
// could be 1.5 times as far off as one rounding of the result alone).  The second term is multiplied
// with the same weights in shared memory.
//
// Measured (bf16, us): gated, 4 rows, 4096 x 8192 (134 MB of weights) 23.5, 5.7 TB/s; input gradient, 16
// rows, 2048 x 8192 (34 MB) 7.5; loss over 32000 x 1024 of 64 rows 15.7, where the pair kernel takes 24.2
// for 65; input gradient of 1024 x 32000 19.3 (23.6).  Gated tiles, 128 columns of two weights for 64 rows, are the
// even point: 4096 x 8192 30.2 (29.5).
//
// Included by exactly one translation unit, after tg_linear_kernel.cuh.
#pragma once

#include "tg_few_config.h"
#include "tg_linear_kernel.cuh"

namespace tg {

struct FewMaps {
  CUtensorMap w[2], x[2], x_rest[2];
};

struct FewParams {
  uint32_t rows, n_pad;              // rows, and as the MMA takes them
  uint32_t terms;                    // 2: x_rest is added to x
  uint32_t outs;                     // results of a row
  uint32_t k_blocks, k_seg;          // of 64; from k_seg on the second maps
  uint32_t tiles, groups;
  float* partials;                   // kEpiStore, groups > 1: [groups][rows][outs]
  uint32_t stages, stage_bytes;
  const float* alpha;                // kEpiStore
  uint32_t act;                      // kEpiGated
  void *out, *g, *u;                 // results; kEpiGated: g and u too, or null
  void* rest;                        // kEpiDlogits: what rounding the results left, or null
  int64_t ld_out, ld_g, ld_u;
  RowWeights loss;                   // kEpiStats: targets; kEpiDlogits: all of it
  uint32_t first_col;                // logits of words first_col ..
  float2* stats;                     // [rows][slots], a slot for each tile
  uint32_t slots;
  float* hit;
  const float* lse;                  // kEpiDlogits
  uint64_t watchdog_ns;
  int64_t inject_skip_phase;
};

struct __align__(8) FewCtl {
  uint64_t loaded[kFewMaxStages];
  uint64_t consumed[kFewMaxStages];
  uint64_t tmem_full[2];
  uint64_t tmem_empty[2];
  uint64_t drain;
  uint32_t filled, filled_par;       // slots that were filled, and the parity of their last fill
  uint32_t tmem_base;
  int abort;
};

__device__ __forceinline__ uint32_t cluster_nctarank() {
  uint32_t n;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(n));
  return n;
}

// As tmem_ld_32x32b_x32, for 16 consecutive columns.
__device__ __forceinline__ void tmem_ld_32x32b_x16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}

// Floats between rows of summed logits: threads with a row each read without bank conflicts.
constexpr uint32_t kStatPitch = kFewM + 1;

// Stores v rounded to 16 bits and gives what it became.
template <int DT>
__device__ __forceinline__ float st_result(void* base, int64_t at, float v) {
  if constexpr (DT == 1) {
    const __nv_bfloat16 r = __float2bfloat16_rn(v);
    static_cast<__nv_bfloat16*>(base)[at] = r;
    return __bfloat162float(r);
  } else {
    const __half r = __float2half_rn(v);
    static_cast<__half*>(base)[at] = r;
    return __half2float(r);
  }
}

// DT: 0 = fp16, 1 = bf16.  W_MN: the weights lie with the results' index contiguous ([k, n]), not k.
template <int DT, int W_MN, int EPI>
__global__ void __launch_bounds__(kFewThreads, 2)
    few_rows_kernel(const __grid_constant__ FewMaps maps, const FewParams p) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ FewCtl ctl;
  constexpr uint32_t kMats = EPI == kEpiGated ? 2u : 1u;
  constexpr uint32_t kChunkBytes = kFewBK * 128u;          // W_MN: 64 rows of 64 columns
  constexpr uint32_t kSegment = kFewSegment<EPI>;
  constexpr bool kParted = kFewParted<EPI>;

  const uint32_t warp = threadIdx.x >> 5;
  const uint32_t lane = threadIdx.x & 31u;
  const uint32_t ranks = cluster_nctarank(), rank = cluster_ctarank();
  const uint32_t unit = blockIdx.x / ranks, group = unit / p.tiles;
  const uint32_t n0 = (unit - group * p.tiles) * kFewM;
  const uint32_t sbase = (smem_u32(smem_raw) + 1023u) & ~1023u;
  const uint32_t stage_bytes = p.stage_bytes;
  const uint32_t per_group = (p.k_blocks + p.groups - 1u) / p.groups;
  const uint32_t g_lo = min(group * per_group, p.k_blocks), g_hi = min(g_lo + per_group, p.k_blocks);
  const uint32_t per_rank = (per_group + ranks - 1u) / ranks;
  const uint32_t k_lo = min(g_lo + rank * per_rank, g_hi), k_hi = min(k_lo + per_rank, g_hi);
  const uint32_t segments = (k_hi - k_lo + kSegment - 1u) / kSegment;

  const uint32_t bar_loaded = smem_u32(&ctl.loaded[0]);
  const uint32_t bar_consumed = smem_u32(&ctl.consumed[0]);
  const uint32_t bar_tmem_full = smem_u32(&ctl.tmem_full[0]);
  const uint32_t bar_tmem_empty = smem_u32(&ctl.tmem_empty[0]);
  const uint32_t bar_drain = smem_u32(&ctl.drain);
  const uint32_t acc_cols = kParted ? kFewRows : kMats * p.n_pad;
  const uint32_t tmem_cols = 2u * acc_cols;                // two accumulators; 32 .. 256

  if (threadIdx.x == 0) {
    for (int s = 0; s < kFewMaxStages; ++s) {
      mbar_init(bar_loaded + 8u * s, 1);
      mbar_init(bar_consumed + 8u * s, 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(bar_tmem_full + 8u * b, 1);
      mbar_init(bar_tmem_empty + 8u * b, kFewEpiThreads / 32);
    }
    mbar_init(bar_drain, 1);
    ctl.abort = 0;
    fence_mbarrier_init();
    prefetch_tensormap(&maps.w[0]);
    if (kMats == 2) prefetch_tensormap(&maps.w[1]);
    prefetch_tensormap(&maps.x[0]);
  }
  __syncwarp();
  if (warp == 1) {
    tmem_alloc(smem_u32(&ctl.tmem_base), tmem_cols);
    tmem_relinquish_alloc_permit();
  }
  tcgen05_fence_before_sync();
  __syncthreads();
  tcgen05_fence_after_sync();
  grid_dependency_wait();      // launched with programmatic stream serialization
  grid_launch_dependents();

  const uint32_t tmem_base = ctl.tmem_base;
  volatile int* abort_flag = &ctl.abort;
  const uint64_t limit = p.watchdog_ns;
  // results of this thread's lane of the accumulator, row by row (epilogue warps)
  float v[kMats][kFewRows];
  // This CTA finishes rows row0 .. row0 + share - 1.  What is read for each (their targets' places
  // among the tile's results, lse, weights) is read ahead: lane i has rows i and i + 32.
  const uint32_t share = p.n_pad / ranks;   // both powers of two
  const uint32_t share_log = 31u - __clz(share);
  const uint32_t row0 = rank * share;
  int32_t hot[2] = {-1, -1};
  float lse[2] = {}, weight[2] = {};
  if constexpr (EPI == kEpiStats || EPI == kEpiDlogits) {
    float top = 0.0f;   // the largest |dloss| of all rows: every warp looks for itself
    if constexpr (EPI == kEpiDlogits) {
      for (uint32_t r = lane; r < p.rows; r += 32u) top = fmaxf(top, p.loss.counted(r));
#pragma unroll
      for (uint32_t o = 16; o > 0; o /= 2) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
      if (blockIdx.x == 0 && threadIdx.x == 0) p.loss.template write_alpha<DT>(top);
    }
#pragma unroll
    for (uint32_t i = 0; i < 2; ++i) {
      const uint32_t r = lane + 32u * i;
      if (warp < 2 || r >= share || row0 + r >= p.rows) continue;
      const int64_t at = p.loss.targets[row0 + r] - static_cast<int64_t>(p.first_col + n0);
      if (at >= 0 && at < kFewM) hot[i] = static_cast<int32_t>(at);
      if constexpr (EPI == kEpiDlogits) {
        lse[i] = p.lse[row0 + r];
        weight[i] = p.loss.template weight<DT>(row0 + r, top);
      }
    }
  }

  if (warp == 0) {
    // ------------------------------------------------------------ TMA producer
    if (lane == 0) {
      uint32_t slot = 0, parity = 0, filled = 0, filled_par = 0;
      // an injected fault: neither its phase nor any after it is filled (a condition around the loads
      // took 0.7 us of 16 k-blocks)
      const uint64_t inject = static_cast<uint64_t>(p.inject_skip_phase);
      const uint32_t k_end = p.inject_skip_phase >= 0 && (inject >> 32) == blockIdx.x
                                 ? min(k_hi, k_lo + static_cast<uint32_t>(inject))
                                 : k_hi;
      for (uint32_t k = k_lo; k < k_end; ++k) {
        if (!wait_or_abort(bar_consumed + 8u * slot, parity ^ 1u, abort_flag, limit,
                           kRoleProducer))
          break;
        const uint32_t bar = bar_loaded + 8u * slot;
        mbar_arrive_expect_tx(bar, stage_bytes);
        const uint32_t seg = k >= p.k_seg ? 1u : 0u;
        const int32_t kx = static_cast<int32_t>(k - seg * p.k_seg) * kFewBK;
        const uint32_t dst = sbase + slot * stage_bytes;
#pragma unroll
        for (uint32_t m = 0; m < kMats; ++m) {
          const CUtensorMap* map = &maps.w[EPI == kEpiGated ? m : seg];
          const uint32_t w_dst = dst + m * kFewWeightBytes;
          if constexpr (W_MN) {
            tma_load_2d(w_dst, map, bar, static_cast<int32_t>(n0), kx);
            tma_load_2d(w_dst + kChunkBytes, map, bar, static_cast<int32_t>(n0) + 64, kx);
          } else {
            tma_load_2d(w_dst, map, bar, kx, static_cast<int32_t>(n0));
          }
        }
        tma_load_2d(dst + kMats * kFewWeightBytes, &maps.x[seg], bar, kx, 0);
        if (p.terms == 2u)
          tma_load_2d(dst + kMats * kFewWeightBytes + p.n_pad * 128u, &maps.x_rest[seg], bar, kx, 0);
        filled |= 1u << slot;
        filled_par = (filled_par & ~(1u << slot)) | (parity << slot);
        if (++slot == p.stages) slot = 0, parity ^= 1u;
      }
      ctl.filled = filled;
      ctl.filled_par = filled_par;
    }
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    const uint32_t idesc = idesc_f16(DT, kFewM, 0, W_MN, 0) | ((p.n_pad >> 3) << 17);
    const bool leader = elect_one();
    const uint64_t a0 = smem_desc_sw128(sbase, W_MN ? kChunkBytes : 16u, 1024);
    const uint64_t b0 = smem_desc_sw128(sbase + kMats * kFewWeightBytes, 16u, 1024);
    uint32_t slot = 0, parity = 0, in_seg = 0, acc = 0, acc_parity = 0;
    for (uint32_t k = k_lo; k < k_hi; ++k) {
      bool got = wait_or_abort(bar_loaded + 8u * slot, parity, abort_flag, limit, kRoleMma);
      if (got && in_seg == 0)   // the accumulator's last segment has been read out
        got = wait_or_abort(bar_tmem_empty + 8u * acc, acc_parity ^ 1u, abort_flag, limit, kRoleMma);
      if (!__all_sync(0xffffffffu, got)) break;
      tcgen05_fence_after_sync();
      if (leader) {
        const uint64_t at = slot * (stage_bytes >> 4);
#pragma unroll
        for (uint32_t m = 0; m < kMats; ++m) {
          const uint32_t d = tmem_base + acc * acc_cols + m * p.n_pad;
#pragma unroll
          for (uint32_t kk = 0; kk < kFewBK / kUmmaK; ++kk) {
            // parted: the steps take turns with the accumulator's parts
            const uint32_t part = kParted ? kk * p.n_pad : 0u;
            const bool add = in_seg != 0u || (kParted ? part >= kFewRows : kk != 0u);
            umma_f16(d + part % kFewRows,
                     a0 + at + m * (kFewWeightBytes >> 4) + (W_MN ? kk * 128u : kk * 2u),
                     b0 + at + kk * 2u, idesc, add ? 1u : 0u);
          }
          if (EPI == kEpiStore && p.terms == 2u) {
#pragma unroll
            for (uint32_t kk = 0; kk < kFewBK / kUmmaK; ++kk)
              umma_f16(d, a0 + at + (W_MN ? kk * 128u : kk * 2u),
                       b0 + at + p.n_pad * 8u + kk * 2u, idesc, 1u);
          }
        }
        umma_commit(bar_consumed + 8u * slot);
      }
      __syncwarp();
      if (++slot == p.stages) slot = 0, parity ^= 1u;
      if (++in_seg == kSegment || k + 1u == k_hi) {
        if (leader) umma_commit(bar_tmem_full + 8u * acc);
        __syncwarp();
        in_seg = 0;
        acc ^= 1u;
        acc_parity ^= acc ^ 1u;
      }
    }
    if (leader) {
      umma_commit(bar_drain);
      wait_bounded(bar_drain, 0, limit, kRoleDrain);
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------ sums of the segments
    const uint32_t q = warp & 3u;
#pragma unroll
    for (uint32_t m = 0; m < kMats; ++m)
#pragma unroll
      for (uint32_t i = 0; i < kFewRows; ++i) v[m][i] = 0.0f;
    uint32_t acc = 0, acc_parity = 0;
    for (uint32_t sg = 0; sg < segments; ++sg) {
      const bool got = wait_or_abort(bar_tmem_full + 8u * acc, acc_parity, abort_flag, limit,
                                     kRoleEpilogue);
      if (!__all_sync(0xffffffffu, got)) break;
      tcgen05_fence_after_sync();
      const uint32_t t_row = tmem_base + ((q * 32u) << 16) + acc * acc_cols;
#pragma unroll
      for (uint32_t m = 0; m < kMats; ++m)
#pragma unroll
        for (uint32_t j = 0; j < kFewRows / 16; ++j) {
          if (!kParted && 16u * j >= p.n_pad) break;
          uint32_t t[16];
          tmem_ld_32x32b_x16(t_row + m * p.n_pad + 16u * j, t);
          auto add_to = [&](uint32_t r) {   // rows r .. r + 15
#pragma unroll
            for (uint32_t i = 0; i < 16; ++i) v[m][r + i] += __uint_as_float(t[i]);
          };
          if (!kParted || p.n_pad == kFewRows) {
            add_to(16 * j);
          } else if (p.n_pad == 32u) {
            add_to(16 * (j & 1u));
          } else {
            add_to(0);
          }
        }
      tcgen05_fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar_tmem_empty + 8u * acc);
      acc ^= 1u;
      acc_parity ^= acc ^ 1u;
    }
  }

  // Every load of this CTA has been multiplied, so the ring is idle; after an abort they are waited for.
  tcgen05_fence_before_sync();
  __syncthreads();
  if (threadIdx.x == 0 && *abort_flag)
    for (uint32_t s = 0; s < p.stages; ++s)
      if ((ctl.filled >> s) & 1u)
        wait_bounded(bar_loaded + 8u * s, (ctl.filled_par >> s) & 1u, limit, kRoleDrain);
  __syncwarp();
  if (warp == 1) {
    tcgen05_fence_after_sync();
    tmem_dealloc(tmem_base, tmem_cols);
  }
  float* const sums = reinterpret_cast<float*>(smem_raw + (sbase - smem_u32(smem_raw)));
  // statistics: the summed logits by rows, behind what the ranks hand out
  float* const stat_rows = sums + (ranks == 1u ? 0u : p.n_pad * kFewM);
  // this thread's result of every row (warps 2..5): its lane of the accumulator
  const uint32_t f = (warp & 3u) * 32u + lane;
  const bool in = n0 + f < p.outs;
  const float alpha = EPI == kEpiStore && p.alpha ? *p.alpha : 1.0f;
  // result f of row row0 + r (b: the up projection's)
  auto finish = [&](uint32_t r, float a, float b) {
    const int64_t row = row0 + r, n = n0 + f;
    if constexpr (EPI == kEpiGated) {
      if (!in) return;
      st_result<DT>(p.out, row * p.ld_out + n, a * gate_of(a, p.act).s * b);
      if (p.g != nullptr) {
        st_result<DT>(p.g, row * p.ld_g + n, a);
        st_result<DT>(p.u, row * p.ld_u + n, b);
      }
    } else if constexpr (EPI == kEpiStore) {
      if (!in) return;
      if (p.partials != nullptr)
        p.partials[(static_cast<int64_t>(group) * p.rows + row) * p.outs + n] = a;
      else
        st_result<DT>(p.out, row * p.ld_out + n, a * alpha);
    } else if constexpr (EPI == kEpiDlogits) {
      const int32_t at = __shfl_sync(0xffffffffu, r < 32u ? hot[0] : hot[1], r & 31u);
      const float row_lse = __shfl_sync(0xffffffffu, r < 32u ? lse[0] : lse[1], r & 31u);
      const float w = __shfl_sync(0xffffffffu, r < 32u ? weight[0] : weight[1], r & 31u);
      float d = exp2_fast((a - row_lse) * kLog2e);
      if (at == static_cast<int32_t>(f)) d -= 1.0f;
      d = w == 0.0f ? 0.0f : d * w;
      if (!in) return;
      const float back = st_result<DT>(p.out, row * p.ld_out + n, d);
      if (p.rest != nullptr) st_result<DT>(p.rest, row * p.ld_out + n, left_over(d, back));
    } else {
      stat_rows[r * kStatPitch + f] = in ? a : -INFINITY;
    }
  };
  if (ranks == 1u) {
    if (warp < 2 || *abort_flag) return;
#pragma unroll
    for (uint32_t i = 0; i < kFewRows; ++i) {
      if (i >= p.rows) break;
      finish(i, v[0][i], v[kMats - 1][i]);
    }
  } else {
    // Sums are handed out by rows: [rank][product][row of the receiver's][128] in the receiver's
    // ring, once all CTAs of the cluster are here.
    cluster_sync();
    if (warp >= 2) {
#pragma unroll
      for (uint32_t m = 0; m < kMats; ++m)
#pragma unroll
        for (uint32_t i = 0; i < kFewRows; ++i) {
          if (i >= p.rows) break;
          const uint32_t to = i >> share_log, r = i & (share - 1u);
          st_shared_cluster_u32(
              mapa_shared(sbase + 4u * (((rank * kMats + m) * share + r) * kFewM + f), to),
              __float_as_uint(v[m][i]));
        }
    }
    cluster_sync();
    if (warp < 2 || *abort_flag) return;
    const uint32_t mine = p.rows > row0 ? min(p.rows - row0, share) : 0u;
    // the ranks' sums in order
#pragma unroll 4
    for (uint32_t r = 0; r < mine; ++r) {
      float t[2] = {0.0f, 0.0f};
      for (uint32_t c = 0; c < ranks; ++c)
#pragma unroll
        for (uint32_t m = 0; m < kMats; ++m)
          t[m] += sums[((c * kMats + m) * share + r) * kFewM + f];
      finish(r, t[0], t[kMats - 1]);
    }
  }
  if constexpr (EPI == kEpiStats) {
    // 128 / share threads to a row, each with every so many'th of its logits, then one joins them
    asm volatile("bar.sync 1, %0;" ::"n"(kFewEpiThreads) : "memory");
    const uint32_t parts = kFewEpiThreads >> share_log;
    const uint32_t r = f & (share - 1u), part = f >> share_log;
    const float* const l = stat_rows + r * kStatPitch;
    float top = -INFINITY, sum = 0.0f;
    const bool row_in = row0 + r < p.rows;
    if (row_in) {
#pragma unroll 8
      for (uint32_t i = part; i < kFewM; i += parts) top = fmaxf(top, l[i]);
      const float base = top == -INFINITY ? 0.0f : top;   // nothing but -inf: exponentials 0
#pragma unroll 8
      for (uint32_t i = part; i < kFewM; i += parts) sum += exp2_fast((l[i] - base) * kLog2e);
    }
    float2* const joint = reinterpret_cast<float2*>(stat_rows + ((share * kStatPitch + 1u) & ~1u));
    joint[f] = make_float2(top, sum);
    asm volatile("bar.sync 1, %0;" ::"n"(kFewEpiThreads) : "memory");
    if (part == 0 && row_in) {
      float m = top;
      for (uint32_t c = 1; c < parts; ++c) m = fmaxf(m, joint[(c << share_log) + r].x);
      const float base = m == -INFINITY ? 0.0f : m;
      float s = 0.0f;
      for (uint32_t c = 0; c < parts; ++c) {
        const float2 j = joint[(c << share_log) + r];
        s += j.y * exp2_fast((j.x - base) * kLog2e);
      }
      const uint64_t row = row0 + r;
      p.stats[row * p.slots + n0 / kFewM] = make_float2(m, s);
      const int32_t at = r < 32u ? hot[0] : hot[1];   // rows r < share: lane r % 32 has them
      if (at >= 0 && n0 + at < p.outs) p.hit[row] = l[at];
    }
  }
}

}  // namespace tg
