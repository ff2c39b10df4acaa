// tg_linear_kernel.cuh -- products with fused epilogues (tcgen05, CTA pairs): what a feed-forward
// block and a vocabulary's cross entropy take from the tensor core, forward and backward.
//
//   D[m, n] = sum_k A[m, k] B[k, n]      fp16 or bf16 in, fp32 accumulation
//
// A lies with k contiguous ("K-major": rows of activations) or with m contiguous ("M-major": the
// transposed activations of a weight gradient, as they lie in memory); B with n contiguous (a weight
// [in, out], or gradients [tokens, out]) or with k contiguous (a weight [in, out] read backwards, or
// the rows of a vocabulary).  No operand is transposed in memory: the MMA takes either.
//
// Two matrices may stand in one operand's place:
//   * gated (kEpiGated): B's columns are the gate's and the up projection's side by side: the even CTA
//     loads 128 of the one, the odd CTA the same 128 of the other, so one MMA gives g in columns 0..127
//     and u in columns 128..255 of each CTA's accumulator, and act(g) u needs no other CTA's data;
//   * along K (k_seg): k-blocks from k_seg on come from the second A and the second B;
//   * along N (n_seg): tiles from n_seg on come from the second B and go to the second C.
// And two products may share a launch (kEpiStore): their units are walked as one list, so that one
// fills the pairs that the other leaves idle (the gradients towards an input and towards its weights).
//
// The pair structure is that of tg_gemm_pair_kernel.cuh; the MMA warp walks its loop together and one
// elected lane issues, as in tg_wgrad_kernel.cuh.  Sums are cut into segments (tg_linear_config.h): eight
// epilogue warps read each out into registers, where the rest of the epilogue happens, so an accumulator
// is free again before anything is stored.  Few tiles: K is split into ranges whose fp32 sums go to a
// workspace [splits][rows rounded up to 32][N], and linear_join_kernel adds them in order.
//
// What bounds it is the tensor pipe, active 84 to 91 % of the time with every epilogue, and back to back
// the card's power: 4096 x 4096 x 65536 with the statistics of a cross entropy 1069 us alone (2.06
// PFLOP/s), 1240 among others at the power cap; input gradient 8192^3 593 and 682.
//
// Included by exactly one translation unit, after tg_wgrad_kernel.cuh.
#pragma once

#include <type_traits>

#include "tg_linear_config.h"
#include "tg_linear_units.h"
#include "tg_wgrad_kernel.cuh"

namespace tg {

// Two products share a launch with kEpiStore only.
template <int EPI>
constexpr int kProducts = EPI == 0 ? 2 : 1;

template <int PRODUCTS>
struct LinearMaps {
  CUtensorMap a[PRODUCTS][2];   // by segment of K
  CUtensorMap b[PRODUCTS][4];   // by segment of N, then of K
  CUtensorMap c[PRODUCTS][3];
};

// The cross entropy's rows: one counts where its target is not ``ignore``; a target outside the
// vocabulary makes NaN of it.
enum TargetKind { kTargetIgnored, kTargetValid, kTargetWrong };
__device__ __forceinline__ TargetKind target_kind(int64_t t, int64_t ignore, uint32_t vocab) {
  if (t == ignore) return kTargetIgnored;
  return t >= 0 && t < static_cast<int64_t>(vocab) ? kTargetValid : kTargetWrong;
}

// The gradient of row r's loss as a weight of its logits' gradients: whole dloss / d where the row counts,
// with d the largest |dloss| of such rows (``top``); 0 for ignored rows, NaN for wrong targets.  alpha = d
// / whole undoes it.  Gradients of logits are so rounded relative to d: where dloss is the same in every
// row, a target's -1 is exact instead of off by one rounding in all rows alike (4096 rows of 65536
// words, bf16: dx 2.9e-3 off, now 1.9e-3; its own rounding makes 1.7e-3).  whole: 1 in bf16; in fp16, which
// has few exponents, 2^15, so that probabilities 2^29 times smaller keep all their bits.
struct RowWeights {
  const float* dloss;
  const int64_t* targets;
  int64_t ignore;
  uint32_t vocab;
  float* alpha;          // written by the first CTA

  __device__ float counted(uint32_t r) const {   // |dloss| of a row that counts, else 0
    return target_kind(targets[r], ignore, vocab) == kTargetValid ? fabsf(dloss[r]) : 0.0f;
  }
  // nothing to be relative to: no gradient at all, or an infinite one
  __device__ static bool plain(float top) { return !(top > 0.0f && top < INFINITY); }
  template <int DT>
  __device__ static constexpr float whole() { return DT == 0 ? 32768.0f : 1.0f; }
  template <int DT>
  __device__ float weight(uint32_t r, float top) const {
    const TargetKind kind = target_kind(targets[r], ignore, vocab);
    if (kind == kTargetWrong) return __int_as_float(0x7fffffff);
    const float d = kind == kTargetValid ? dloss[r] : 0.0f;
    return plain(top) ? d : d / top * whole<DT>();
  }
  template <int DT>
  __device__ void write_alpha(float top) const { *alpha = plain(top) ? 1.0f : top / whole<DT>(); }
};

struct LinearParams : LinearWalk {
  uint32_t act, keep;                // kEpiGated: the activation; 1: g and u are stored as well
  // cross entropy: logits of columns first_col .. of the vocabulary
  uint32_t first_col, slots;
  float2* stats;                     // kEpiStats: [M][slots] maximum, sum of exponentials
  float* hit;                        // kEpiStats: [M] the target's logit
  const float* lse;                  // kEpiDlogits: [M]
  RowWeights rows;                   // targets; the rest for kEpiDlogits
  uint64_t watchdog_ns;
  int64_t inject_skip_phase;
};

struct __align__(8) LinearCtl {
  uint64_t loaded[kLinStages];       // used in the even CTA only
  uint64_t consumed[kLinStages];
  uint64_t tmem_full[2];             // accumulators: columns 0..255 and 256..511 of TMEM
  uint64_t tmem_empty[2];            // used in the even CTA only
  uint64_t drain;
  uint64_t odd_done;
  PairFills<kLinStages> fills;
  uint32_t sink[kLinEpiWarps];
  float top[kLinEpiWarps];           // kEpiDlogits: the warps' largest |dloss|
  uint32_t tmem_base;
  int abort;
};

// The logistic function's value s at z(g) and z'(g): act(g) = g s, act'(g) = s + g s (1 - s) z'.
// SiLU: z = g.  GELU (tanh form): z = 2 sqrt(2 / pi) (g + 0.044715 g^3); past |g| = 16 its s is 0 or 1
// in fp32, so g is held there and its cube stays finite.
struct Gate {
  float s, slope;
};
__device__ __forceinline__ Gate gate_of(float g, uint32_t act) {
  float z = g, slope = 1.0f;
  if (act != 0) {
    const float h = fminf(fmaxf(g, -16.0f), 16.0f), h2 = h * h;
    z = 1.5957691216f * fmaf(0.044715f * h2, h, h);
    slope = 1.5957691216f * fmaf(3.0f * 0.044715f, h2, 1.0f);
    if (g != g) z = g;
  }
  return {__fdividef(1.0f, 1.0f + __expf(-z)), slope};
}

// 2-D tiled reduction shared -> global: fp32 values are added to what is there.
__device__ __forceinline__ void tma_add_2d(const CUtensorMap* map, uint32_t src, int32_t x,
                                           int32_t y) {
  asm volatile(
      "cp.reduce.async.bulk.tensor.2d.global.shared::cta.add.tile.bulk_group [%0, {%2, %3}], [%1];" ::
          "l"(reinterpret_cast<uint64_t>(map)),
      "r"(src), "r"(x), "r"(y)
      : "memory");
}

constexpr float kLog2e = 1.4426950408889634f;

// 2^x, by the special-function unit (0 below 2^-126)
__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

template <int N>
__device__ __forceinline__ void registers_down() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void registers_up() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}

// Stores 32 rows x 64 columns of 16-bit results (pk: lane = row) at row0, x by the warp's staging
// buffer and the TMA, which clips at the matrix's edge.
__device__ __forceinline__ void linear_store_packed(const uint32_t (&pk)[32], uint32_t lane,
                                                    uint32_t sbuf, const CUtensorMap* map,
                                                    int32_t row0, int32_t x, uint32_t m,
                                                    uint32_t n) {
  if (lane == 0) bulk_wait_group_read<0>();   // the buffer's last store has read it
  __syncwarp();
#pragma unroll
  for (uint32_t c = 0; c < 8; ++c)
    st_shared_v4(sbuf + lane * 128u + ((c ^ (lane & 7u)) << 4), pk[4 * c], pk[4 * c + 1],
                 pk[4 * c + 2], pk[4 * c + 3]);
  fence_proxy_async_shared();
  __syncwarp();
  if (lane == 0) {
    if (row0 < static_cast<int32_t>(m) && x < static_cast<int32_t>(n))
      tma_store_2d(map, sbuf, x, row0);
    bulk_commit_group();
  }
  __syncwarp();
}

// The same for 32 columns of fp32 sums, stored or added.
__device__ __forceinline__ void linear_store_sums(const float* v, uint32_t lane, uint32_t sbuf,
                                                  const CUtensorMap* map, int32_t row0, bool in,
                                                  int32_t x, uint32_t n, bool add) {
  if (lane == 0) bulk_wait_group_read<0>();
  __syncwarp();
#pragma unroll
  for (uint32_t c = 0; c < 8; ++c)
    st_shared_v4(sbuf + lane * 128u + ((c ^ (lane & 7u)) << 4), __float_as_uint(v[4 * c]),
                 __float_as_uint(v[4 * c + 1]), __float_as_uint(v[4 * c + 2]),
                 __float_as_uint(v[4 * c + 3]));
  fence_proxy_async_shared();
  __syncwarp();
  if (lane == 0) {
    if (in && x < static_cast<int32_t>(n)) {
      if (add)
        tma_add_2d(map, sbuf, x, row0);
      else
        tma_store_2d(map, sbuf, x, row0);
    }
    bulk_commit_group();
  }
  __syncwarp();
}

// What rounding v to ``back`` left; nothing where that overflowed.
__device__ __forceinline__ float left_over(float v, float back) {
  return fabsf(back) == INFINITY ? 0.0f : v - back;
}

template <int DT>
__device__ __forceinline__ void pack64(const float* v, uint32_t (&pk)[32]) {
#pragma unroll
  for (uint32_t i = 0; i < 32; ++i)
    pk[i] = pack_out<DT>(__float_as_uint(v[2 * i]), __float_as_uint(v[2 * i + 1]));
}

// DT: 0 = fp16, 1 = bf16.
template <int DT, int EPI>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kLinThreads, 1)
    linear_pair_kernel(const __grid_constant__ LinearMaps<kProducts<EPI>> maps,
                       const __grid_constant__ LinearParams p) {
  extern __shared__ uint8_t smem_raw[];
  constexpr uint32_t kStages = kLinStages, kStageBytes = kLinStageBytes;
  constexpr uint32_t kOperand = kLinOperandBytes;
  constexpr uint32_t kAtomBytes = kBM * 128u;              // K-major: 128 rows of 128 bytes
  constexpr uint32_t kChunkBytes = kLinBK * 128u;          // MN-major: kLinBK rows of 64 columns
  constexpr int kTile = EPI == kEpiGated ? kGatedTileN : kBN;
  // which way an operand lies: any with kEpiStore, one way with the other epilogues
  auto a_lies_mn = [](const LinearProblem& q) { return EPI == kEpiStore && q.a_mn != 0u; };
  auto b_lies_mn = [](const LinearProblem& q) {
    return EPI == kEpiGated || (EPI == kEpiStore && q.b_mn != 0u);
  };
  // and how long its segments are: logits that are stored as parts have shorter ones than results
  auto segment_log_of = [](const LinearProblem& q) {
    return EPI == kEpiStore   ? q.segment_log
           : EPI == kEpiGated ? kLinSegmentLog
                              : kLogitSegmentLog;
  };
  __shared__ LinearCtl ctl;

  const uint32_t warp = threadIdx.x >> 5;
  const uint32_t lane = threadIdx.x & 31u;
  const uint32_t rank = cluster_ctarank();
  const uint32_t pair = blockIdx.x >> 1;
  const uint32_t num_pairs = gridDim.x >> 1;
  const uint32_t sbase = (smem_u32(smem_raw) + 1023u) & ~1023u;
  const uint32_t sA0 = sbase;                      // stage s: A, then B
  const uint32_t sB0 = sA0 + kOperand;
  const uint32_t sEpi = sbase + kStages * kStageBytes;

  const uint32_t bar_loaded = smem_u32(&ctl.loaded[0]);
  const uint32_t bar_consumed = smem_u32(&ctl.consumed[0]);
  const uint32_t bar_tmem_full = smem_u32(&ctl.tmem_full[0]);
  const uint32_t bar_tmem_empty = smem_u32(&ctl.tmem_empty[0]);
  const uint32_t bar_drain = smem_u32(&ctl.drain);

  if (threadIdx.x == 0) {
#pragma unroll
    for (uint32_t s = 0; s < kStages; ++s) {
      mbar_init(bar_loaded + 8u * s, 1);
      mbar_init(bar_consumed + 8u * s, 1);
      ctl.fills.par[s] = 0;
    }
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      mbar_init(bar_tmem_full + 8u * b, 1);
      mbar_init(bar_tmem_empty + 8u * b, kLinEpiWarps);
    }
    mbar_init(bar_drain, 1);
    mbar_init(smem_u32(&ctl.odd_done), 1);
    ctl.abort = 0;
    fence_mbarrier_init();
  }
  if (warp == 0 && lane == 0) {
    prefetch_tensormap(&maps.a[0][0]);
    prefetch_tensormap(&maps.b[0][EPI == kEpiGated ? rank : 0u]);
    if (EPI != kEpiStats) prefetch_tensormap(&maps.c[0][0]);
    if (EPI == kEpiStore && p.units[1] != 0u) {
      prefetch_tensormap(&maps.a[kProducts<EPI> - 1][0]);
      prefetch_tensormap(&maps.b[kProducts<EPI> - 1][0]);
      prefetch_tensormap(&maps.c[kProducts<EPI> - 1][0]);
    }
  }
  __syncwarp();
  if (warp == 2) {
    tmem_alloc_pair(smem_u32(&ctl.tmem_base), kTmemCols);
    tmem_relinquish_alloc_permit_pair();
  }
  tcgen05_fence_before_sync();
  cluster_sync();   // both CTAs' barriers exist before any remote arrive or complete_tx
  tcgen05_fence_after_sync();
  grid_dependency_wait();      // launched with programmatic stream serialization
  grid_launch_dependents();

  const uint32_t tmem_base = ctl.tmem_base;
  volatile int* abort_flag = &ctl.abort;
  const uint32_t peer_abort = mapa_shared(smem_u32(&ctl.abort), rank ^ 1u);
  const uint64_t limit = p.watchdog_ns;

  if (warp < kFirstEpiWarp) {
    registers_down<kLinFewRegs>();
    if (warp == 0) {
      // ---------------------------------------------------------- TMA producer (both CTAs)
      if (lane == 0) {
        bool ok = true;
        uint64_t phase = 0;
        RingPos<kStages> at;
        for (LinearUnits<kProducts<EPI>> un(p, pair, num_pairs); ok && un.valid(); un.next()) {
          const PersistentTileScheduler& sched = un.sched;
          const LinearProblem& q = un.q();
          const bool a_mn = a_lies_mn(q), b_mn = b_lies_mn(q);
          const bool half = sched.half_unit();
          const uint32_t seg_n = sched.n_idx >= q.n_seg ? 1u : 0u;
          const int32_t nt = static_cast<int32_t>(sched.n_idx - seg_n * q.n_seg);
          const int32_t m0 = static_cast<int32_t>(sched.m_idx * kPairBM + rank * kBM);
          // this CTA's first column (gated: the same columns of the gate's matrix in the even CTA, of
          // the up projection's in the odd one)
          const int32_t own = EPI == kEpiGated ? 0 : static_cast<int32_t>(rank) * (half ? 64 : 128);
          const int32_t n0 = nt * kTile + (half ? sched.part * (kTile / 2) : 0) + own;
          // a half-width unit's B with columns contiguous is one chunk of 64; of rows of K all 128
          // rows are loaded and the MMA reads 64
          const uint32_t b_chunks = b_mn && half ? 1u : 2u;
          const uint32_t own_bytes = kOperand + b_chunks * (kOperand / 2u);
          const uint32_t k_seg = q.k_seg;
          const CUtensorMap* const maps_a = &maps.a[un.product()][0];
          const CUtensorMap* const maps_b = &maps.b[un.product()][EPI == kEpiGated ? rank : seg_n];
          for (uint32_t k = un.k_lo; k < un.k_hi; ++k, ++phase, at.advance(1)) {
            const uint32_t s = at.slot, par = at.parity;
            if (!pair_wait_or_abort(bar_consumed + 8u * s, par ^ 1u, abort_flag, peer_abort, limit,
                                    kRoleProducer)) {
              ok = false;
              break;
            }
            if (injected_skip(p.inject_skip_phase, phase))
              continue;  // injected fault: this CTA never arms or fills this phase
            const uint32_t full_even = mapa_shared(bar_loaded + 8u * s, 0);
            if (rank == 0) mbar_arrive_expect_tx(bar_loaded + 8u * s, 2u * own_bytes);
            const uint32_t seg_k = k >= k_seg ? 1u : 0u;
            const int32_t kx = static_cast<int32_t>(k - seg_k * k_seg) * kLinBK;
            const CUtensorMap* tmA = maps_a + seg_k;
            const CUtensorMap* tmB = maps_b + 2u * seg_k;
            const uint32_t a_dst = sA0 + s * kStageBytes, b_dst = sB0 + s * kStageBytes;
            // two boxes of 16 KiB each: 64-column chunks, or 64-deep atoms of K
#pragma unroll
            for (uint32_t c = 0; c < 2; ++c) {
              const int32_t on = static_cast<int32_t>(c * 64u);
              tma_load_2d_pair(a_dst + c * kAtomBytes, tmA, full_even, a_mn ? m0 + on : kx + on,
                               a_mn ? kx : m0);
            }
#pragma unroll
            for (uint32_t c = 0; c < 2; ++c) {
              const int32_t on = static_cast<int32_t>(c * 64u);
              if (c < b_chunks)
                tma_load_2d_pair(b_dst + c * kAtomBytes, tmB, full_even, b_mn ? n0 + on : kx + on,
                                 b_mn ? kx : n0);
            }
            record_fill(ctl.fills, s, phase, par, own_bytes);
          }
        }
        // the odd producer has stopped filling: its records are final (see pair_drain_fills)
        if (rank == 1) mbar_arrive_cluster(mapa_shared(smem_u32(&ctl.odd_done), 0));
      }
      __syncwarp();
    } else if (warp == 1) {
      // ---------------------------------------------------------- MMA issuer (even CTA)
      if (rank == 0) {
        constexpr uint32_t idesc_full = idesc_f16(DT, kPairBM, kBN, 0, 0);
        constexpr uint32_t idesc_half = idesc_f16(DT, kPairBM, kBN / 2, 0, 0);
        const bool leader = elect_one();
        bool ok = true;
        RingPos<kStages> ring;
        RingPos<2> acc;                 // the accumulator of the next segment
        // a descriptor is an addition to the low word of a constant one (the address field: 16-byte
        // units, below 2^14)
        const uint64_t k_desc = smem_desc_sw128(sA0, 16u, 1024);
        const uint64_t mn_desc = smem_desc_sw128(sA0, kChunkBytes, 1024);
        const uint32_t hi = static_cast<uint32_t>(k_desc >> 32);   // the same for both
        auto commit = [&](uint32_t bar) {
          if (leader) umma_commit_pair_multicast(bar, 0x3);
          __syncwarp();
        };
        auto wait = [&](uint32_t bar, uint32_t parity) {
          const bool got = pair_wait_or_abort<true>(bar, parity, abort_flag, peer_abort, limit,
                                                    kRoleMma);
          return __all_sync(0xffffffffu, got) != 0;
        };
        // One unit.  How the operands lie is fixed in each copy of the loop: descriptors that had to
        // be chosen between in it made the MMAs wait (input gradient 8192^3 597 -> 606 us).
        auto unit = [&](const LinearUnits<kProducts<EPI>>& un, auto a_mn, auto b_mn) {
          constexpr bool A = decltype(a_mn)::value, B = decltype(b_mn)::value;
          // where K-step kk (16 deep) begins: 16 rows of 128 bytes on, or 32 bytes on within an atom
          auto step = [](bool mn, uint32_t kk) {
            return mn ? kk * 128u : (kk / 4u) * (kAtomBytes >> 4) + (kk % 4u) * 2u;
          };
          const uint32_t idesc = (un.sched.half_unit() ? idesc_half : idesc_full) |
                                 (A ? 1u << 15 : 0u) | (B ? 1u << 16 : 0u);
          const uint32_t a_lo = static_cast<uint32_t>(A ? mn_desc : k_desc);
          const uint32_t b_lo = static_cast<uint32_t>(B ? mn_desc : k_desc) + (kOperand >> 4);
          const uint32_t nk = un.k_hi - un.k_lo, segment = 1u << segment_log_of(un.q());
          uint32_t in_seg = 0;          // k-blocks of the segment so far
          for (uint32_t k = 0; k < nk; ++k, ring.advance(1)) {
            const uint32_t s = ring.slot;
            // both CTAs' epilogues have read the accumulator's last segment out
            if (!wait(bar_loaded + 8u * s, ring.parity) ||
                (in_seg == 0 && !wait(bar_tmem_empty + 8u * acc.slot, acc.parity ^ 1u)))
              return false;
            tcgen05_fence_after_sync();
            const uint32_t d = tmem_base + acc.slot * kBN;
            const uint32_t at = s * (kStageBytes >> 4);
            if (leader) {
#pragma unroll
              for (uint32_t kk = 0; kk < kLinBK / kUmmaK; ++kk)
                umma_f16_pair_words(d, a_lo + at + step(A, kk), hi, b_lo + at + step(B, kk), hi,
                                    idesc, in_seg != 0u || kk != 0u ? 1u : 0u);
            }
            commit(bar_consumed + 8u * s);
            if (++in_seg == segment || k + 1 == nk) {
              commit(bar_tmem_full + 8u * acc.slot);
              acc.advance(1);
              in_seg = 0;
            }
          }
          return true;
        };
        using No = std::false_type;
        using Yes = std::true_type;
        for (LinearUnits<kProducts<EPI>> un(p, pair, num_pairs); ok && un.valid(); un.next()) {
          if constexpr (EPI == kEpiStore)
            ok = un.q().a_mn   ? unit(un, Yes(), Yes())
                 : un.q().b_mn ? unit(un, No(), Yes())
                               : unit(un, No(), No());
          else if constexpr (EPI == kEpiGated)
            ok = unit(un, No(), Yes());
          else
            ok = unit(un, No(), No());
        }
        if (leader) {
          umma_commit_pair_multicast(bar_drain, 0x1);
          wait_bounded(bar_drain, 0, limit, kRoleDrain);
        }
      }
      __syncwarp();
    }
  } else {
    // ------------------------------------------------------------ epilogue (both CTAs)
    registers_up<kLinEpiRegs>();
    const uint32_t e = warp - kFirstEpiWarp, q = e & 3u, side = e >> 2;
    const uint32_t sink_even = mapa_shared(smem_u32(&ctl.sink[e]), 0);
    const uint32_t sbuf = sEpi + e * kEpiBufBytes;
    // read once: in every unit it kept the stores waiting
    const float alphas[2] = {EPI == kEpiStore && p.q[0].alpha ? *p.q[0].alpha : 1.0f,
                             EPI == kEpiStore && p.q[1].alpha ? *p.q[1].alpha : 1.0f};
    float row_top = 0.0f;   // kEpiDlogits: the largest |dloss| of all rows
    if constexpr (EPI == kEpiDlogits) {
      const uint32_t tt = threadIdx.x - 32u * kFirstEpiWarp;
      for (uint32_t r = tt; r < p.q[0].M; r += 32u * kLinEpiWarps)
        row_top = fmaxf(row_top, p.rows.counted(r));
#pragma unroll
      for (uint32_t o = 16; o > 0; o /= 2)
        row_top = fmaxf(row_top, __shfl_xor_sync(0xffffffffu, row_top, o));
      if (lane == 0) ctl.top[e] = row_top;
      asm volatile("bar.sync 1, %0;" ::"n"(32 * kLinEpiWarps) : "memory");
#pragma unroll
      for (int o = 0; o < kLinEpiWarps; ++o) row_top = fmaxf(row_top, ctl.top[o]);
      if (blockIdx.x == 0 && tt == 0) p.rows.template write_alpha<DT>(row_top);
    }
    RingPos<2> acc;
    bool ok = true;
    for (LinearUnits<kProducts<EPI>> un(p, pair, num_pairs); ok && un.valid(); un.next()) {
      const PersistentTileScheduler& sched = un.sched;
      const LinearProblem& o = un.q();
      const CUtensorMap* const maps_c = &maps.c[un.product()][0];
      const bool half = sched.half_unit();      // the accumulator has 128 columns
      const uint32_t seg_n = sched.n_idx >= o.n_seg ? 1u : 0u;
      const int32_t nt = static_cast<int32_t>(sched.n_idx - seg_n * o.n_seg);
      const int32_t row0 = static_cast<int32_t>(sched.m_idx * kPairBM + rank * kBM + q * 32u);
      const uint32_t row = static_cast<uint32_t>(row0) + lane;
      const bool row_in = row < o.M;
      // this warp's columns of the accumulator, 64 at a time: two chunks, or one of a half unit's.
      // Gated: one of g and the one of u that goes with it; of a half unit's single one side 0 takes
      // both
      uint32_t chunks, c0, c1;
      int32_t x0;
      const int32_t tile0 = nt * kTile + (half ? sched.part * (kTile / 2) : 0);
      if constexpr (EPI == kEpiGated) {
        chunks = half && side ? 0u : 2u;
        c0 = half ? 0u : side;
        c1 = half ? 1u : 2u + side;
        x0 = tile0 + static_cast<int32_t>(c0) * kEpiN;
      } else {
        chunks = half ? 1u : 2u;
        c0 = half ? side : 2u * side;
        c1 = c0 + 1u;
        x0 = tile0 + static_cast<int32_t>(c0) * kEpiN;
      }
      // the sums of all segments: columns of chunk c0, then of c1
      float v[128];
      const uint32_t nk = un.k_hi - un.k_lo;
      const uint32_t segments = ((nk - 1u) >> segment_log_of(o)) + 1u;
#pragma unroll 1
      for (uint32_t sg = 0; sg < segments; ++sg, acc.advance(1)) {
        const bool got = pair_wait_or_abort(bar_tmem_full + 8u * acc.slot, acc.parity, abort_flag,
                                            peer_abort, limit, kRoleEpilogue);
        if (!__all_sync(0xffffffffu, got)) {
          ok = false;
          break;
        }
        tcgen05_fence_after_sync();
        const uint32_t t_row = tmem_base + ((q * 32u) << 16) + acc.slot * kBN;
        if (sg == 0) {
#pragma unroll
          for (uint32_t j = 0; j < 4; ++j) {
            if (j / 2u >= chunks) break;
            uint32_t t[32];
            tmem_ld_32x32b_x32(t_row + (j < 2 ? c0 : c1) * kEpiN + (j & 1u) * 32u, t);
#pragma unroll
            for (uint32_t i = 0; i < 32; ++i) v[32 * j + i] = __uint_as_float(t[i]);
          }
        } else {
#pragma unroll
          for (uint32_t j = 0; j < 4; ++j) {
            if (j / 2u >= chunks) break;
            uint32_t t[32];
            tmem_ld_32x32b_x32(t_row + (j < 2 ? c0 : c1) * kEpiN + (j & 1u) * 32u, t);
#pragma unroll
            for (uint32_t i = 0; i < 32; ++i) v[32 * j + i] += __uint_as_float(t[i]);
          }
        }
        tcgen05_fence_before_sync();
        pair_report_warp(bar_tmem_empty + 8u * acc.slot, rank, lane, sink_even);
      }
      if (!ok) break;
      if constexpr (EPI == kEpiGated) {
        if (chunks) {
          uint32_t pk[32];
          if (p.keep) {
            pack64<DT>(v, pk);
            linear_store_packed(pk, lane, sbuf, maps_c + 1, row0, x0, o.M, o.N);
            pack64<DT>(v + 64, pk);
            linear_store_packed(pk, lane, sbuf, maps_c + 2, row0, x0, o.M, o.N);
          }
          // from the unrounded g and u
#pragma unroll
          for (uint32_t i = 0; i < 64; ++i) v[i] = v[i] * gate_of(v[i], p.act).s * v[64 + i];
          pack64<DT>(v, pk);
          linear_store_packed(pk, lane, sbuf, maps_c, row0, x0, o.M, o.N);
        }
      } else if constexpr (EPI == kEpiStore) {
        if (o.partial) {
          const int32_t to = static_cast<int32_t>(un.split * o.part_rows) + row0;
          const bool in = row0 < static_cast<int32_t>(o.M);
#pragma unroll
          for (uint32_t j = 0; j < 4; ++j) {
            if (j / 2u >= chunks) break;
            linear_store_sums(v + 32 * j, lane, sbuf, maps_c + seg_n, to, in,
                              x0 + static_cast<int32_t>(32u * j), o.N, o.partial == 2);
          }
        } else {
          if (o.alpha) {
            const float alpha = un.product() == 0u ? alphas[0] : alphas[1];
#pragma unroll
            for (uint32_t i = 0; i < 128; ++i) v[i] *= alpha;
          }
#pragma unroll
          for (uint32_t j = 0; j < 2; ++j) {
            if (j >= chunks) break;
            uint32_t pk[32];
            pack64<DT>(v + 64 * j, pk);
            linear_store_packed(pk, lane, sbuf, maps_c + seg_n, row0,
                                x0 + static_cast<int32_t>(64u * j), o.M, o.N);
          }
        }
      } else {
        // the target's place among this warp's columns, or a place that none of them has
        // (differences from x0: x0 + 128 may be 2^31)
        const uint64_t hot =
            row_in ? static_cast<uint64_t>(p.rows.targets[row]) - p.first_col - static_cast<uint64_t>(x0)
                   : 128u;
        const int32_t at = hot < 128u ? static_cast<int32_t>(hot) : -1;
        if constexpr (EPI == kEpiStats) {
          const int32_t left = static_cast<int32_t>(o.N) - x0;   // words from x0 on
          if (chunks == 1 || left < 128) {
            // columns that another warp has, or past the vocabulary
            const int32_t end = min(static_cast<int32_t>(64u * chunks), left);
#pragma unroll
            for (uint32_t i = 0; i < 128; ++i)
              if (static_cast<int32_t>(i) >= end) v[i] = -INFINITY;
          }
          if (__any_sync(0xffffffffu, at >= 0)) {
            float l = 0.0f;
#pragma unroll
            for (uint32_t i = 0; i < 128; ++i)
              if (static_cast<int32_t>(i) == at) l = v[i];
            if (at >= 0 && at < static_cast<int32_t>(64u * chunks)) p.hit[row] = l;
          }
          // maximum and sum; a NaN goes through the sum
          float m4[4] = {v[0], v[1], v[2], v[3]};
#pragma unroll
          for (uint32_t i = 4; i < 128; ++i) m4[i & 3u] = fmaxf(m4[i & 3u], v[i]);
          const float top = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3]));
          const float base = top == -INFINITY ? 0.0f : top;   // nothing but -inf: exponentials 0
          float s4[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
          for (uint32_t i = 0; i < 128; ++i) s4[i & 3u] += exp2_fast((v[i] - base) * kLog2e);
          // slots of 64 columns; two chunks leave the second one's empty
          if (row_in && x0 < static_cast<int32_t>(o.N)) {
            const uint32_t slot = static_cast<uint32_t>(x0) / kStatCols;
            float2* to = p.stats + static_cast<uint64_t>(row) * p.slots + slot;
            to[0] = make_float2(top, (s4[0] + s4[1]) + (s4[2] + s4[3]));
            if (chunks == 2 && slot + 1u < p.slots) to[1] = make_float2(-INFINITY, 0.0f);
          }
        } else {
          const float lse = row_in ? p.lse[row] : 0.0f;
          const float weight = row_in ? p.rows.template weight<DT>(row, row_top) : 0.0f;
#pragma unroll
          for (uint32_t j = 0; j < 2; ++j) {
            if (j >= chunks) break;
#pragma unroll
            for (uint32_t i = 64 * j; i < 64 * j + 64; ++i) {
              float d = exp2_fast((v[i] - lse) * kLog2e);
              if (static_cast<int32_t>(i) == at) d -= 1.0f;
              v[i] = weight == 0.0f ? 0.0f : d * weight;
            }
            uint32_t pk[32];
            pack64<DT>(v + 64 * j, pk);
            linear_store_packed(pk, lane, sbuf, maps_c, row0,
                                x0 + static_cast<int32_t>(64u * j), o.M, o.N);
          }
        }
      }
    }
    // the stores have read shared memory; the grid's end makes them visible
    if (lane == 0) bulk_wait_group_read<0>();
    __syncwarp();
  }

  __syncthreads();   // every role of this CTA has left its loop
  if (rank == 0 && warp == 0 && lane == 0 && *abort_flag)
    pair_drain_fills(bar_loaded, ctl.fills, mapa_shared(smem_u32(&ctl.fills), 1),
                     smem_u32(&ctl.odd_done), limit);
  tcgen05_fence_before_sync();
  cluster_sync();   // neither CTA leaves while the pair may still touch its smem or TMEM
  if (warp == 2) {
    tcgen05_fence_after_sync();
    tmem_dealloc_pair(tmem_base, kTmemCols);
  }
}

// out = alpha times the sum of the splits' partial sums [splits][part_rows][cols], in order, rounded
// once.  A thread takes 4 neighbouring columns of a row (cols is a multiple of 4) and reads four splits
// at a time.  One launch joins what one launch of products left (blockIdx.y).
struct JoinParams {
  const float* partials;
  const float* alpha;
  void* out;
  int64_t ld_out;
  uint64_t stride4;          // float4s between splits
  uint32_t splits, rows, cols;
};
struct JoinJobs {
  JoinParams job[3];
};
template <int DT>
__global__ void __launch_bounds__(256) linear_join_kernel(const __grid_constant__ JoinJobs jobs) {
  grid_dependency_wait();
  grid_launch_dependents();
  const JoinParams& p = jobs.job[blockIdx.y];
  const float f = p.alpha ? *p.alpha : 1.0f;
  const uint32_t vecs = p.cols / 4u;
  const uint64_t total = static_cast<uint64_t>(p.rows) * vecs, stride4 = p.stride4;
  for (uint64_t i = static_cast<uint64_t>(blockIdx.x) * blockDim.x + threadIdx.x; i < total;
       i += static_cast<uint64_t>(gridDim.x) * blockDim.x) {
    const uint64_t row = i / vecs;
    const uint32_t v = static_cast<uint32_t>(i - row * vecs);
    const float4* src = reinterpret_cast<const float4*>(p.partials) + i;
    float4 a = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    uint32_t s = 0;
    for (; s + 4u <= p.splits; s += 4u, src += 4u * stride4) {
      float4 c[4];
#pragma unroll
      for (uint32_t j = 0; j < 4; ++j) c[j] = __ldcg(src + j * stride4);
#pragma unroll
      for (uint32_t j = 0; j < 4; ++j) a.x += c[j].x, a.y += c[j].y, a.z += c[j].z, a.w += c[j].w;
    }
    for (; s < p.splits; ++s, src += stride4) {
      const float4 c = __ldcg(src);
      a.x += c.x, a.y += c.y, a.z += c.z, a.w += c.w;
    }
    uint2 o;
    o.x = pack_out<DT>(__float_as_uint(a.x * f), __float_as_uint(a.y * f));
    o.y = pack_out<DT>(__float_as_uint(a.z * f), __float_as_uint(a.w * f));
    *reinterpret_cast<uint2*>(static_cast<char*>(p.out) +
                              (static_cast<int64_t>(row) * p.ld_out + 4ll * v) * 2) = o;
  }
}

}  // namespace tg
