// tg_wgrad_kernel.cuh -- the weight gradient taken from an 8-bit checkpoint (tcgen05, CTA pairs).
//
//   dW[i, n] = sum over tokens t of x[t, i] dY[t, n],   x[t, i] = q[t, i] 2^(s[t, i/32] - 127)
//
// A GEMM whose contraction runs over the rows of both operands: A = x^T [cols, tokens] and B = dY
// [tokens, outs] both lie with their M resp. N index contiguous, which the MMA takes as MN-major
// operands; neither is transposed in memory.  The checkpoint is read as it is, one byte a value, and
// becomes 16-bit in shared memory: E4M3 has 4 significant bits, so x is exact in bf16 and fp16
// (rounded once where it leaves their range), products are exact and sums are fp32.
//
// The pair structure is that of tg_gemm_pair_kernel.cuh and, for tiles of two N-halves (256 x 512),
// of tg_gemm_pair_wide_kernel.cuh: CTA r holds columns 128 r .. of x as its rows of A, and half of
// each N-half's columns of dY.  One more role: per k-block of 64 tokens warp 3 loads 64 x 128 bytes
// of q and their scales into a ring of their own, and warps 8.., four to a k-block,
// turn them into the A operand (two chunks of 64 columns x 64 tokens, 128-byte swizzle) and report
// to the even CTA's ``made`` barrier (there also for the dY bytes of both CTAs), which the MMA
// thread waits for.
//
// What bounds it: with two N-halves the tensor pipe and the power cap, 8192^3 at 1882 to 1971 TFLOP/s
// (the dense GEMM reaches 1980); the MMAs of a k-block take 1024 cycles, and the widening's reads and
// writes of 8 + 16 KiB go on behind them.  With one N-half shared memory: a k-block moves about 656
// wavefronts for 512 cycles of MMAs (32768 x 1000 x 512, 37 us).
//
// Few tiles: the tokens are split into ``splits`` ranges, (tile, range) units write fp32 partial
// sums to a workspace [splits][m_blocks * 256][outs], and wgrad_join_kernel adds them in order.
//
// Included by exactly one translation unit, after tg_gemm_pair_kernel.cuh.
#pragma once

#include "tg_gemm_pair_kernel.cuh"
#include "tg_rows.cuh"
#include "tg_wgrad_config.h"

namespace tg {

struct WgradParams : GemmParams {   // M = cols, N = outs, K = tokens
  const uint8_t* scales;            // [tokens][scale_cols]
  uint32_t scale_cols;
  uint32_t tma_scales;              // 1: rows of scales are whole 16-byte units (tmS)
  uint32_t splits, blocks_per_split;
};

// One worker's walk over units u = worker + w * workers: the tile units of every split in turn.
struct WgradUnits {
  PersistentTileScheduler sched;
  uint32_t u, w, step, units, per_split, kps, k_blocks;
  uint32_t split, k_lo, k_hi;

  __device__ WgradUnits(const WgradParams& p, uint32_t worker, uint32_t workers)
      : sched(p.m_blocks, p.n_blocks, p.group, workers, p.split_from, p.total_units,
              p.column_major),
        u(worker), w(0), step(workers), units(p.total_units * p.splits), per_split(p.total_units),
        kps(p.blocks_per_split), k_blocks(p.k_blocks) {
    decode();
  }
  __device__ bool valid() const { return u < units; }
  __device__ void next() {
    u += step;
    ++w;
    decode();
  }
  __device__ void decode() {
    if (u >= units) return;
    split = u / per_split;
    sched.jump(u - split * per_split, w);
    k_lo = split * kps;
    k_hi = k_lo + kps < k_blocks ? k_lo + kps : k_blocks;
  }
};

template <int NH>
struct __align__(8) WgradCtl {
  using Cfg = WgradConfig<NH>;
  uint64_t loaded[Cfg::kStages];     // dY boxes of both CTAs; used in the even CTA only
  uint64_t made[Cfg::kStages];       // and the A operand as well; used in the even CTA only
  uint64_t consumed[Cfg::kStages];
  uint64_t raw_full[Cfg::kRaws];     // this CTA's checkpoint bytes
  uint64_t scale_full[Cfg::kRaws];   // and their scales
  uint64_t raw_empty[Cfg::kRaws];    // both are in registers
  uint64_t tmem_full[2];             // accumulators: columns 0..255 and 256..511 of TMEM
  uint64_t tmem_empty[2];            // used in the even CTA only
  uint64_t drain;
  uint64_t odd_done;
  PairFills<Cfg::kStages> fills;
  uint32_t sink[kEpiWarps + Cfg::kGroups * kWgMakeWarps];
  uint32_t tmem_base;
  int abort;
};

// Asynchronous copy of ``bytes`` (0..4) bytes to shared memory, the rest of the 4 zero-filled; both
// addresses 4-byte aligned.
__device__ __forceinline__ void cp_async_4(uint32_t dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(bytes)
               : "memory");
}

// Arrives on ``bar`` (one of its initial count) once this thread's copies so far have landed.
__device__ __forceinline__ void cp_async_arrive(uint32_t bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}

__device__ __forceinline__ void cp_async_wait_all() {
  asm volatile("cp.async.wait_all;" ::: "memory");
}

__device__ __forceinline__ uint32_t ld_shared_u8(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}

__device__ __forceinline__ void st_shared_u8(uint32_t addr, uint32_t v) {
  asm volatile("st.shared.u8 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}

// umma_f16_pair with the descriptors given as two words each.
__device__ __forceinline__ void umma_f16_pair_words(uint32_t d_tmem, uint32_t a_lo, uint32_t a_hi,
                                                    uint32_t b_lo, uint32_t b_hi, uint32_t idesc,
                                                    uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\t"
      "mov.b64 a, {%1, %2};\n\t"
      "mov.b64 b, {%3, %4};\n\t"
      "setp.ne.b32 p, %6, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], a, b, %5, p;\n\t}" ::"r"(d_tmem),
      "r"(a_lo), "r"(a_hi), "r"(b_lo), "r"(b_hi), "r"(idesc), "r"(accumulate)
      : "memory");
}

// One lane of the warp, the same at every call; every lane calls it.
__device__ __forceinline__ bool elect_one() {
  uint32_t leader;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.b32 %0, 1, 0, p;\n\t}"
      : "=r"(leader));
  return leader != 0;
}

// A position in a ring of N slots and the parity of its present turn.
template <uint32_t N>
struct RingPos {
  uint32_t slot = 0, parity = 0;
  __device__ __forceinline__ void advance(uint32_t by) {   // by <= N
    slot += by;
    if (slot >= N) {
      slot -= N;
      parity ^= 1u;
    }
  }
};

// 16 E4M3 bytes times 2^(s - 127), to 16-bit values packed in pairs; exact but for the final
// rounding, any bytes.
template <int DT>
__device__ __forceinline__ void widen_any(const uint32_t (&in)[4], uint32_t s, uint32_t (&out)[8]) {
  const float scale = e8m0_value(s);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float2 f = e4m3x2_value((in[i / 2] >> (16 * (i & 1))) & 0xFFFFu);
    out[i] = pack_out<DT>(__float_as_uint(f.x * scale), __float_as_uint(f.y * scale));
  }
}

// The same by moving bits: E4M3's exponent and fraction put in the place of the 16-bit type's read
// as the value times 2^-120 (bf16) or 2^-8 (fp16), subnormals included, and one multiplication by
// 2^(s - 7) or 2^(s - 119) sets that right with one rounding.  Right unless a byte is NaN or the
// factor is not a number of the type (s > 134; fp16 also s < 95): ``top`` gathers the largest
// magnitudes as they were moved, in both halves, for widened_right.
template <int DT>
__device__ __forceinline__ void widen_short(const uint32_t (&in)[4], uint32_t s, uint32_t (&out)[8],
                                            uint32_t& top) {
  uint32_t factor;   // the power of two in both halves
  if constexpr (DT == 1) {
    factor = (s + 120u) << 7;
  } else {
    factor = s >= 105u ? (s - 104u) << 10 : 1u << (s - 95u);
  }
  factor = __byte_perm(factor, 0u, 0x1010u);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    // bytes 2 (i % 2) and + 1 of the word to the high bytes of the two halves
    const uint32_t t = __byte_perm(in[i / 2], 0u, i & 1 ? 0x3424u : 0x1404u);
    if constexpr (DT == 1) {
      const uint32_t m = (t >> 4) & 0x07F007F0u;
      const uint32_t b = (t & 0x80008000u) | m;
      top = __vmaxu2(top, m);
      const __nv_bfloat162 r = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&b),
                                       *reinterpret_cast<const __nv_bfloat162*>(&factor));
      out[i] = *reinterpret_cast<const uint32_t*>(&r);
    } else {
      const uint32_t m = (t >> 1) & 0x3F803F80u;
      const uint32_t b = (t & 0x80008000u) | m;
      top = __vmaxu2(top, m);
      const __half2 r = __hmul2(*reinterpret_cast<const __half2*>(&b),
                                *reinterpret_cast<const __half2*>(&factor));
      out[i] = *reinterpret_cast<const uint32_t*>(&r);
    }
  }
}

// Whether widen_short was right for all that went into ``top`` and for scales s_min .. s_max.
template <int DT>
__device__ __forceinline__ bool widened_right(uint32_t top, uint32_t s_min, uint32_t s_max) {
  constexpr uint32_t nan = DT == 1 ? 0x07F0u : 0x3F80u;   // E4M3 NaN, moved
  return (top & 0xFFFFu) < nan && (top >> 16) < nan && s_max <= 134u && (DT == 1 || s_min >= 95u);
}

// Stores one 64-column chunk of the accumulator (v: lane = row, fp32 bits) as fp32 partial sums,
// 32 columns at a time through the warp's two staging buffers; tmP clips columns, and every row of
// a tile has a place.
__device__ __forceinline__ void wgrad_store_partial(const uint32_t (&v)[64], uint32_t lane,
                                                    uint32_t sbuf0, const CUtensorMap* tmP,
                                                    int32_t row0, int32_t x, uint32_t n) {
#pragma unroll
  for (uint32_t h = 0; h < 2; ++h) {
    const uint32_t sbuf = sbuf0 + h * kEpiBufBytes;
    if (lane == 0) bulk_wait_group_read<1>();   // the store that last read this buffer is done
    __syncwarp();
#pragma unroll
    for (uint32_t c = 0; c < 8; ++c)
      st_shared_v4(sbuf + lane * 128u + ((c ^ (lane & 7u)) << 4), v[32 * h + 4 * c],
                   v[32 * h + 4 * c + 1], v[32 * h + 4 * c + 2], v[32 * h + 4 * c + 3]);
    fence_proxy_async_shared();
    __syncwarp();
    if (lane == 0) {
      const int32_t xh = x + static_cast<int32_t>(32 * h);
      if (xh < static_cast<int32_t>(n)) tma_store_2d(tmP, sbuf, xh, row0);
      bulk_commit_group();
    }
  }
  __syncwarp();
}

// DT: 0 = fp16, 1 = bf16 (dY and dW).  NH: N-halves per tile.  SPLIT: partial sums to the workspace
// (tmC is then the workspace's map).  DEBUG adds fault injection.
template <int DT, int NH, bool SPLIT, bool DEBUG>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(WgradConfig<NH>::kThreads, 1)
    wgrad_pair_kernel(const __grid_constant__ CUtensorMap tmQ,
                      const __grid_constant__ CUtensorMap tmB,
                      const __grid_constant__ CUtensorMap tmC,
                      const __grid_constant__ CUtensorMap tmS, const WgradParams p) {
  extern __shared__ uint8_t smem_raw[];
  using Cfg = WgradConfig<NH>;
  constexpr uint32_t kStages = Cfg::kStages, kRaws = Cfg::kRaws, kStageBytes = Cfg::kStageBytes;
  __shared__ WgradCtl<NH> ctl;

  const uint32_t warp = threadIdx.x >> 5;
  const uint32_t lane = threadIdx.x & 31u;
  const uint32_t rank = cluster_ctarank();
  const uint32_t pair = blockIdx.x >> 1;
  const uint32_t num_pairs = gridDim.x >> 1;
  const uint32_t sbase = (smem_u32(smem_raw) + 1023u) & ~1023u;
  const uint32_t sA0 = sbase;                      // stage s: A, then dY chunks (2 h + c)
  const uint32_t sB0 = sA0 + kWgABytes;
  const uint32_t sR0 = sbase + kStages * kStageBytes;
  const uint32_t sEpi = sR0 + kRaws * kWgRawBytes;
  const uint32_t sS0 = sEpi + kEpiSmemBytes;       // scales of raw slot r: sS0 + r * kWgScaleBytes

  const uint32_t bar_loaded = smem_u32(&ctl.loaded[0]);
  const uint32_t bar_made = smem_u32(&ctl.made[0]);
  const uint32_t bar_consumed = smem_u32(&ctl.consumed[0]);
  const uint32_t bar_raw_full = smem_u32(&ctl.raw_full[0]);
  const uint32_t bar_scale_full = smem_u32(&ctl.scale_full[0]);
  const uint32_t bar_raw_empty = smem_u32(&ctl.raw_empty[0]);
  const uint32_t bar_tmem_full = smem_u32(&ctl.tmem_full[0]);
  const uint32_t bar_tmem_empty = smem_u32(&ctl.tmem_empty[0]);
  const uint32_t bar_drain = smem_u32(&ctl.drain);

  if (threadIdx.x == 0) {
#pragma unroll
    for (uint32_t s = 0; s < kStages; ++s) {
      mbar_init(bar_loaded + 8u * s, 1);
      mbar_init(bar_made + 8u * s, kWgMakeWarps);
      mbar_init(bar_consumed + 8u * s, 1);
      ctl.fills.par[s] = 0;
    }
#pragma unroll
    for (uint32_t r = 0; r < kRaws; ++r) {
      mbar_init(bar_raw_full + 8u * r, 1);
      mbar_init(bar_scale_full + 8u * r, 32);
      mbar_init(bar_raw_empty + 8u * r, kWgMakeWarps);
    }
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      mbar_init(bar_tmem_full + 8u * b, 1);
      mbar_init(bar_tmem_empty + 8u * b, kEpiWarps);
    }
    mbar_init(bar_drain, 1);
    mbar_init(smem_u32(&ctl.odd_done), 1);
    ctl.abort = 0;
    fence_mbarrier_init();
  }
  if (warp == 0 && lane == 0) {
    prefetch_tensormap(&tmQ);
    prefetch_tensormap(&tmB);
    prefetch_tensormap(&tmC);
    if (p.tma_scales) prefetch_tensormap(&tmS);
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

  if (warp == 0) {
    // ------------------------------------------------------------ dY loads (both CTAs)
    if (lane == 0) {
      bool ok = true;
      uint64_t phase = 0;
      RingPos<kStages> at;
      for (WgradUnits un(p, pair, num_pairs); ok && un.valid(); un.next()) {
        const PersistentTileScheduler& sched = un.sched;
        const bool half = sched.half_unit();
        // chunks of 64 columns this CTA loads, and the first column of each N-half's share
        const uint32_t chunks = half ? NH : 2u * NH;
        const int32_t n0 =
            static_cast<int32_t>(sched.n_idx) * Cfg::kTileN +
            (half ? sched.part * (Cfg::kTileN / 2) : 0) +
            static_cast<int32_t>(rank) * (half && NH == 1 ? kPairBNHalf / 2 : kPairBNHalf);
        const uint32_t tx_bytes = 2u * chunks * kWgChunkBytes;
        for (uint32_t k = un.k_lo; k < un.k_hi; ++k, ++phase, at.advance(1)) {
          const uint32_t s = at.slot, par = at.parity;
          if (!pair_wait_or_abort(bar_consumed + 8u * s, par ^ 1u, abort_flag, peer_abort, limit,
                                  kRoleProducer)) {
            ok = false;
            break;
          }
          if (DEBUG && injected_skip(p.inject_skip_phase, phase))
            continue;  // injected fault: this CTA never arms or fills this phase
          const int32_t kx = static_cast<int32_t>(k) * kWgBK;
          const uint32_t full_even = mapa_shared(bar_loaded + 8u * s, 0);
          if (rank == 0) mbar_arrive_expect_tx(bar_loaded + 8u * s, tx_bytes);
#pragma unroll
          for (uint32_t c = 0; c < 2u * NH; ++c) {
            if (c >= chunks) break;
            tma_load_2d_pair(sB0 + s * kStageBytes + c * kWgChunkBytes, &tmB, full_even,
                             n0 + static_cast<int32_t>((c / 2u) * kBN + (c % 2u) * kBChunkCols),
                             kx);
          }
          record_fill(ctl.fills, s, phase, par, tx_bytes / 2u);
        }
      }
      // the odd producer has stopped filling: its records are final (see pair_drain_fills)
      if (rank == 1) mbar_arrive_cluster(mapa_shared(smem_u32(&ctl.odd_done), 0));
    }
    __syncwarp();
  } else if (warp == 3) {
    // ------------------------------------------------------------ checkpoint loads (both CTAs)
    if (lane == 0) {
      uint32_t pending = 0, pending_par = 0;   // fills that may still be in flight
      bool ok = true;
      RingPos<kRaws> at;
      for (WgradUnits un(p, pair, num_pairs); ok && un.valid(); un.next()) {
        const int32_t m0 = static_cast<int32_t>(un.sched.m_idx * kPairBM + rank * kBM);
        // scales by TMA: 16 neighbouring bytes of each token's row, from a 16-byte boundary on
        const int32_t sc = (m0 / kCkptBlock) & ~15;
        for (uint32_t k = un.k_lo; k < un.k_hi; ++k, at.advance(1)) {
          const uint32_t r = at.slot, par = at.parity;
          if (!pair_wait_or_abort(bar_raw_empty + 8u * r, par ^ 1u, abort_flag, peer_abort, limit,
                                  kRoleProducer)) {
            ok = false;
            break;
          }
          const int32_t kx = static_cast<int32_t>(k) * kWgBK;
          mbar_arrive_expect_tx(bar_raw_full + 8u * r,
                                kWgRawBytes + (p.tma_scales ? kWgScaleBytes : 0u));
          tma_load_2d(sR0 + r * kWgRawBytes, &tmQ, bar_raw_full + 8u * r, m0, kx);
          if (p.tma_scales)
            tma_load_2d(sS0 + r * kWgScaleBytes, &tmS, bar_raw_full + 8u * r, sc, kx);
          pending |= 1u << r;
          pending_par = (pending_par & ~(1u << r)) | (par << r);
        }
      }
      if (!ok) {
        for (uint32_t r = 0; r < kRaws; ++r)
          if ((pending >> r) & 1u)
            wait_bounded(bar_raw_full + 8u * r, (pending_par >> r) & 1u, limit, kRoleDrain);
      }
    }
    __syncwarp();
  } else if (warp == 2) {
    // ------------------------------------------------------------ scale loads (both CTAs)
    // A lane takes tokens lane and lane + 32 of the k-block: the 4 scales of this CTA's 128 columns
    // start at byte o of the scale array, and are copied with the 4-byte words around them, so
    // scale j lies at byte o % 4 + j of the token's place.  Bytes past the array's end are zero-filled.
    // (Past the row's end they are the next row's, and multiply zeros.)  An array that does not
    // start on a 4-byte boundary is read byte by byte, without running ahead.  Where rows of scales
    // are whole 16-byte units warp 3 loads them by TMA instead, one box a k-block: these copies
    // take a shared-memory cycle for each word (8192^3: 678 us with them, 640 without).
    const bool words = (reinterpret_cast<uintptr_t>(p.scales) & 3u) == 0u;
    const uint64_t total = static_cast<uint64_t>(p.K) * p.scale_cols;
    bool ok = !p.tma_scales;
    RingPos<kRaws> ring;
    for (WgradUnits un(p, pair, num_pairs); ok && un.valid(); un.next()) {
      const uint32_t sc = (un.sched.m_idx * kPairBM + rank * kBM) / kCkptBlock;
      for (uint32_t k = un.k_lo; k < un.k_hi; ++k, ring.advance(1)) {
        const uint32_t r = ring.slot, par = ring.parity;
        const bool got = pair_wait_or_abort(bar_raw_empty + 8u * r, par ^ 1u, abort_flag,
                                            peer_abort, limit, kRoleProducer);
        if (!__all_sync(0xffffffffu, got)) {
          ok = false;
          break;
        }
#pragma unroll
        for (uint32_t i = 0; i < 2; ++i) {
          const uint32_t row = i * 32u + lane;
          const uint64_t o = (static_cast<uint64_t>(k) * kWgBK + row) * p.scale_cols + sc;
          const uint32_t dst = sS0 + r * kWgScaleBytes + row * kWgScalePitch;
          if (words) {
#pragma unroll
            for (uint32_t h = 0; h < 2; ++h) {
              const uint64_t at = (o & ~3ull) + 4u * h;
              const uint64_t left = at < total ? total - at : 0;
              cp_async_4(dst + 4u * h, p.scales + (left ? at : 0),
                         static_cast<uint32_t>(left < 4 ? left : 4));
            }
          } else {
#pragma unroll
            for (uint32_t j = 0; j < 4; ++j)
              st_shared_u8(dst + (o & 3u) + j, o + j < total ? p.scales[o + j] : 0u);
          }
        }
        if (words)
          cp_async_arrive(bar_scale_full + 8u * r);
        else
          mbar_arrive(bar_scale_full + 8u * r);
      }
    }
    cp_async_wait_all();
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer (even CTA)
    // The whole warp walks the loop and one elected lane issues: control flow and operands are then
    // uniform, which the instruction wants; a single lane on its own copied each operand over, and
    // its 90 cycles an MMA bounded the kernel (k-blocks of four MMAs took 810 cycles).
    if (rank == 0) {
      constexpr uint32_t idesc_full = idesc_f16(DT, kPairBM, kBN, /*A M-major*/ 1, /*B N-major*/ 1);
      constexpr uint32_t idesc_half = idesc_f16(DT, kPairBM, kBN / 2, 1, 1);
      const bool leader = elect_one();
      bool ok = true;
      RingPos<kStages> ring;
      uint32_t uses[2] = {0, 0};      // units that have used each accumulator
      // a descriptor is an addition to the low word of a constant one (the address field: 16-byte
      // units, below 2^14)
      const uint64_t a0 = smem_desc_sw128(sA0, kWgChunkBytes, 1024);
      const uint64_t b0 = smem_desc_sw128(sB0, kWgChunkBytes, 1024);
      const uint32_t a_lo = static_cast<uint32_t>(a0), b_lo = static_cast<uint32_t>(b0);
      const uint32_t a_hi = static_cast<uint32_t>(a0 >> 32), b_hi = static_cast<uint32_t>(b0 >> 32);
      // MMAs of N-half h into accumulator ``acc`` for the k-block in ring slot s
      auto issue_half = [&](uint32_t s, uint32_t h, uint32_t acc, bool first, uint32_t idesc) {
        const uint32_t at = s * (kStageBytes >> 4), d = tmem_base + acc * kBN;
        const uint32_t a = a_lo + at, b = b_lo + at + h * (2u * kWgChunkBytes >> 4);
        if (leader) {
#pragma unroll
          for (uint32_t kk = 0; kk < kWgBK / kUmmaK; ++kk)   // 16 tokens = 2048 bytes on
            umma_f16_pair_words(d, a + kk * 128u, a_hi, b + kk * 128u, b_hi, idesc,
                                !first || kk != 0u ? 1u : 0u);
        }
      };
      auto commit = [&](uint32_t bar) {
        if (leader) umma_commit_pair_multicast(bar, 0x3);
        __syncwarp();
      };
      auto wait = [&](uint32_t bar, uint32_t parity) {
        const bool got = pair_wait_or_abort<true>(bar, parity, abort_flag, peer_abort, limit,
                                                  kRoleMma);
        return __all_sync(0xffffffffu, got) != 0;
      };
      auto acc_free = [&](uint32_t acc) {   // both CTAs' epilogues have read its last unit out
        const bool got = wait(bar_tmem_empty + 8u * acc, (uses[acc] & 1u) ^ 1u);
        ++uses[acc];
        tcgen05_fence_after_sync();
        return got;
      };
      for (WgradUnits un(p, pair, num_pairs); ok && un.valid(); un.next()) {
        const bool half = un.sched.half_unit();
        const uint32_t halves = half ? 1u : NH;
        const uint32_t acc0 = NH == 1 ? un.w & 1u : 0u;
        const uint32_t idesc = half && NH == 1 ? idesc_half : idesc_full;
        const uint32_t nk = un.k_hi - un.k_lo;
        // N-half 1 of the first k-block waits until the epilogue has handed accumulator 1 back;
        // that slot is released once both halves have read it
        const uint32_t defer = halves == 2u && nk > 1u ? 1u : 0u;
        const uint32_t s0 = ring.slot;
        for (uint32_t k = 0; k < nk; ++k, ring.advance(1)) {
          const uint32_t s = ring.slot;
          if (!wait(bar_made + 8u * s, ring.parity) || (k == 0 && !acc_free(acc0))) {
            ok = false;
            break;
          }
          tcgen05_fence_after_sync();
          issue_half(s, 0, acc0, k == 0, idesc);
          if (halves == 2u) {
            if (k < defer) continue;
            if (k == defer) {
              if (!acc_free(1)) {
                ok = false;
                break;
              }
              if (defer) {   // catch N-half 1 up
                issue_half(s0, 1, 1, true, idesc);
                commit(bar_consumed + 8u * s0);
              }
            }
            issue_half(s, 1, 1, k == 0, idesc);
          }
          commit(bar_consumed + 8u * s);
        }
        if (!ok) break;
        commit(bar_tmem_full + 8u * acc0);
        if (halves == 2u) commit(bar_tmem_full + 8u);
      }
      if (leader) {
        umma_commit_pair_multicast(bar_drain, 0x1);
        wait_bounded(bar_drain, 0, limit, kRoleDrain);
      }
    }
    __syncwarp();
  } else if (warp >= kWgFirstMakeWarp) {
    // ------------------------------------------------------------ checkpoint bytes -> A operand
    // Group g takes k-blocks g, g + groups, ...  Eight threads take a token's 128 bytes, 16 each;
    // the group's threads cover 16 tokens at a time.  A warp reads 512 neighbouring bytes; a thread
    // writes its 32 bytes as two 16-byte chunks of the token's row of column chunk c / 4, and the
    // threads of column chunk 1 write their second one first, so that eight threads never meet in
    // a bank.
    const uint32_t group = (warp - kWgFirstMakeWarp) / kWgMakeWarps;
    const uint32_t tt = threadIdx.x - (kWgFirstMakeWarp + group * kWgMakeWarps) * 32u;
    const uint32_t c = tt & 7u, r0 = tt >> 3;
    const uint32_t sink_even = mapa_shared(smem_u32(&ctl.sink[warp - kFirstEpiWarp]), 0);
    const bool swap = c >= 4u;
    // where the thread's two chunks of token row r0 go (r0 + 16 i has the same r % 8)
    const uint32_t base = (c / 4u) * kWgChunkBytes + r0 * 128u;
    const uint32_t at0 = base + (((2u * (c & 3u) + (swap ? 1u : 0u)) ^ (r0 & 7u)) << 4);
    const uint32_t at1 = base + (((2u * (c & 3u) + (swap ? 0u : 1u)) ^ (r0 & 7u)) << 4);
    RingPos<kStages> ring;
    RingPos<kRaws> raw;
    ring.advance(group);
    raw.advance(group);
    uint32_t skip = group;   // k-blocks of the units ahead until this group's next one
    bool ok = true;
    for (WgradUnits un(p, pair, num_pairs); ok && un.valid(); un.next()) {
      const uint32_t nk = un.k_hi - un.k_lo;
      // this thread's scale of token r0: by TMA at the unit's place in its 16 bytes, else at byte
      // o % 4 (the same for r0 + 16 i in every k-block)
      const uint32_t sc = (un.sched.m_idx * kPairBM + rank * kBM) / kCkptBlock;
      const uint32_t scale_at = sS0 + r0 * kWgScalePitch + c / 2u +
                                (p.tma_scales ? sc & 15u : (r0 * p.scale_cols) & 3u);
      uint32_t k = skip;
      for (; k < nk; k += Cfg::kGroups, ring.advance(Cfg::kGroups), raw.advance(Cfg::kGroups)) {
        const uint32_t r = raw.slot, s = ring.slot;
        bool got = pair_wait_or_abort(bar_raw_full + 8u * r, raw.parity, abort_flag, peer_abort,
                                      limit, kRoleProducer) &&
                   (p.tma_scales ||
                    pair_wait_or_abort(bar_scale_full + 8u * r, raw.parity, abort_flag, peer_abort,
                                       limit, kRoleProducer));
        if (!__all_sync(0xffffffffu, got)) {
          ok = false;
          break;
        }
        uint32_t in[kWgPasses][4], scale[kWgPasses];
#pragma unroll
        for (uint32_t i = 0; i < kWgPasses; ++i) {
          ld_shared_v4(sR0 + r * kWgRawBytes + (i * 16u + r0) * 128u + c * 16u, in[i][0], in[i][1],
                       in[i][2], in[i][3]);
          scale[i] = ld_shared_u8(scale_at + r * kWgScaleBytes + i * 16u * kWgScalePitch);
        }
#pragma unroll
        for (uint32_t i = 0; i < kWgPasses; ++i) {
          // the half that is written first comes first
          const uint32_t w0 = in[i][0], w1 = in[i][1];
          in[i][0] = swap ? in[i][2] : w0;
          in[i][1] = swap ? in[i][3] : w1;
          in[i][2] = swap ? w0 : in[i][2];
          in[i][3] = swap ? w1 : in[i][3];
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(bar_raw_empty + 8u * r);   // the bytes are in registers
        got = pair_wait_or_abort(bar_consumed + 8u * s, ring.parity ^ 1u, abort_flag, peer_abort,
                                 limit, kRoleProducer);
        if (!__all_sync(0xffffffffu, got)) {
          ok = false;
          break;
        }
        const uint32_t a = sA0 + s * kStageBytes;
        auto put = [&](uint32_t i, const uint32_t (&out)[8]) {
          st_shared_v4(a + at0 + i * 2048u, out[0], out[1], out[2], out[3]);
          st_shared_v4(a + at1 + i * 2048u, out[4], out[5], out[6], out[7]);
        };
        uint32_t top = 0, s_min = 255, s_max = 0;
#pragma unroll
        for (uint32_t i = 0; i < kWgPasses; ++i) {
          uint32_t out[8];
          widen_short<DT>(in[i], scale[i], out, top);
          put(i, out);
          s_min = min(s_min, scale[i]);
          s_max = max(s_max, scale[i]);
        }
        if (!widened_right<DT>(top, s_min, s_max)) {   // rare: again, the long way
#pragma unroll
          for (uint32_t i = 0; i < kWgPasses; ++i) {
            uint32_t out[8];
            widen_any<DT>(in[i], scale[i], out);
            put(i, out);
          }
        }
        __syncwarp();
        fence_proxy_async_shared();
        // the report of the even CTA's first warp of the group also says that dY has landed, so
        // the MMA thread has one barrier to wait for (two took it 100 cycles more a k-block)
        if (rank == 0 && tt < 32u) {
          got = pair_wait_or_abort(bar_loaded + 8u * s, ring.parity, abort_flag, peer_abort, limit,
                                   kRoleProducer);
          if (!__all_sync(0xffffffffu, got)) {
            ok = false;
            break;
          }
        }
        pair_report_warp(bar_made + 8u * s, rank, lane, sink_even);
      }
      skip = k - nk;
    }
    __syncwarp();
  } else if (warp >= kFirstEpiWarp) {
    // ------------------------------------------------------------ epilogue (both CTAs)
    const uint32_t q = warp - kFirstEpiWarp;
    const uint32_t sink_even = mapa_shared(smem_u32(&ctl.sink[q]), 0);
    uint32_t chunk = 0;
    uint32_t uses[2] = {0, 0};
    bool ok = true;
    for (WgradUnits un(p, pair, num_pairs); ok && un.valid(); un.next()) {
      const bool half = un.sched.half_unit();
      const uint32_t halves = half ? 1u : NH;
      const uint32_t chunks = half && NH == 1 ? kBN / kEpiN / 2 : kBN / kEpiN;
      const int32_t row0 =
          static_cast<int32_t>(un.sched.m_idx * kPairBM + rank * kBM + q * 32u);
#pragma unroll 1
      for (uint32_t h = 0; h < halves; ++h) {
        const uint32_t acc = NH == 1 ? un.w & 1u : h;
        const bool got = pair_wait_or_abort(bar_tmem_full + 8u * acc, uses[acc] & 1u, abort_flag,
                                            peer_abort, limit, kRoleEpilogue);
        if (!__all_sync(0xffffffffu, got)) {
          ok = false;
          break;
        }
        ++uses[acc];
        tcgen05_fence_after_sync();
        const int32_t col0 = static_cast<int32_t>(un.sched.n_idx) * Cfg::kTileN +
                             (half ? un.sched.part * (Cfg::kTileN / 2) : 0) +
                             static_cast<int32_t>(h) * kBN;
        const uint32_t t_row = tmem_base + ((q * 32u) << 16) + acc * kBN;
#pragma unroll 1
        for (uint32_t j = 0; j < chunks; ++j, ++chunk) {
          uint32_t v[64];
          tmem_ld_32x32b_x64(t_row + j * kEpiN, v);
          if (j == chunks - 1) {
            tcgen05_fence_before_sync();
            pair_report_warp(bar_tmem_empty + 8u * acc, rank, lane, sink_even);
          }
          const int32_t x = col0 + static_cast<int32_t>(j * kEpiN);
          if constexpr (SPLIT) {
            wgrad_store_partial(v, lane, sEpi + q * 2u * kEpiBufBytes, &tmC,
                                static_cast<int32_t>(un.split * p.m_blocks * kPairBM) + row0, x,
                                p.N);
          } else {
            epilogue_store_chunk<DT>(v, lane, sEpi + (q * 2u + (chunk & 1u)) * kEpiBufBytes, &tmC,
                                     p, row0, x);
          }
        }
      }
    }
    if (lane == 0) bulk_wait_group<0>();
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

// dW = the sum of the splits' partial sums [splits][part_rows][outs], in order, rounded once.  A
// thread takes 4 neighbouring columns of a row (outs is a multiple of 8) and reads four splits at a
// time, so that what bounds it is the L2's bandwidth and not a chain of reads.
template <int DT>
__global__ void __launch_bounds__(256)
    wgrad_join_kernel(const float* __restrict__ partials, uint32_t splits, uint64_t split_stride,
                      uint32_t rows, uint32_t outs, void* __restrict__ dw, int64_t ld_dw) {
  grid_dependency_wait();
  grid_launch_dependents();
  const uint32_t vecs = outs / 4u;
  const uint64_t total = static_cast<uint64_t>(rows) * vecs, stride4 = split_stride / 4u;
  for (uint64_t i = static_cast<uint64_t>(blockIdx.x) * blockDim.x + threadIdx.x; i < total;
       i += static_cast<uint64_t>(gridDim.x) * blockDim.x) {
    const uint32_t row = static_cast<uint32_t>(i / vecs), v = static_cast<uint32_t>(i % vecs);
    const float4* src = reinterpret_cast<const float4*>(partials) + i;
    float4 a = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    uint32_t s = 0;
    for (; s + 4u <= splits; s += 4u, src += 4u * stride4) {
      float4 c[4];
#pragma unroll
      for (uint32_t j = 0; j < 4; ++j) c[j] = __ldcg(src + j * stride4);
#pragma unroll
      for (uint32_t j = 0; j < 4; ++j) a.x += c[j].x, a.y += c[j].y, a.z += c[j].z, a.w += c[j].w;
    }
    for (; s < splits; ++s, src += stride4) {
      const float4 c = __ldcg(src);
      a.x += c.x, a.y += c.y, a.z += c.z, a.w += c.w;
    }
    uint2 o;
    o.x = pack_out<DT>(__float_as_uint(a.x), __float_as_uint(a.y));
    o.y = pack_out<DT>(__float_as_uint(a.z), __float_as_uint(a.w));
    *reinterpret_cast<uint2*>(static_cast<char*>(dw) +
                              (static_cast<int64_t>(row) * ld_dw + 4 * v) * 2) = o;
  }
}

}  // namespace tg
