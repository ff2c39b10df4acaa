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
// The pair structure is that of tg_gemm_pair_kernel.cuh (256 x 256 tiles, CTA r holding columns
// 128 r .. of x as its rows of A, and half of the tile's columns of dY) with one more role: per
// k-block of 64 tokens the producer loads 64 x 128 bytes of q (``raw``) and the dY boxes, warps
// 8..11 turn the bytes into the A operand (two chunks of 64 columns x 64 tokens, 128-byte swizzle)
// and report to the even CTA's ``made`` barrier, and the MMA thread waits for both CTAs' reports
// and dY bytes.  Turning 8192 bytes a k-block takes each of the 128 threads 64 values, about half
// of the 512 cycles that the MMAs of the k-block take.
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

struct __align__(8) WgradCtl {
  uint64_t loaded[kWgStages];        // dY boxes of both CTAs; used in the even CTA only
  uint64_t made[kWgStages];          // A operand of both CTAs; used in the even CTA only
  uint64_t raw[kWgStages];           // this CTA's checkpoint bytes
  uint64_t consumed[kWgStages];
  uint64_t tmem_full[2];
  uint64_t tmem_empty[2];            // used in the even CTA only
  uint64_t drain;
  uint64_t odd_done;
  PairFills<kWgStages> fills;
  uint32_t sink[kEpiWarps + kWgMakeWarps];
  uint32_t tmem_base;
  int abort;
};

// 16 E4M3 bytes times 2^(s - 127), to 16-bit values packed in pairs; exact but for the final
// rounding, any bytes.
template <int DT>
__device__ __noinline__ void widen_any(const uint32_t (&in)[4], uint32_t s, uint32_t (&out)[8]) {
  const float scale = e8m0_value(s);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float2 f = e4m3x2_value((in[i / 2] >> (16 * (i & 1))) & 0xFFFFu);
    out[i] = pack_out<DT>(__float_as_uint(f.x * scale), __float_as_uint(f.y * scale));
  }
}

// The same for bytes without NaN and scales up to 2^7, by moving bits: E4M3's exponent and fraction
// put in the place of the 16-bit type's read as the value times 2^-120 (bf16) or 2^-8 (fp16),
// subnormals included, and one multiplication by 2^(s - 7) or 2^(s - 119) sets that right with one
// rounding.  Larger scales, where that factor would leave the type (and fp16's below 2^-24, s < 95),
// and NaN go the long way.
template <int DT>
__device__ __forceinline__ void widen16(const uint32_t (&in)[4], uint32_t s, uint32_t (&out)[8]) {
  uint32_t nan = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) nan |= ((in[i] & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u;
  if (nan != 0u || s > 134u || (DT == 0 && s < 95u)) {
    widen_any<DT>(in, s, out);
    return;
  }
  uint32_t factor;   // the power of two in both halves
  if constexpr (DT == 1) {
    factor = (s + 120u) << 7;
  } else {
    factor = s >= 105u ? (s - 104u) << 10 : 1u << (s - 95u);
  }
  factor |= factor << 16;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    // bytes 2 (i % 2) and + 1 of the word to the high bytes of the two halves
    const uint32_t t = __byte_perm(in[i / 2], 0u, i & 1 ? 0x3424u : 0x1404u);
    if constexpr (DT == 1) {
      const uint32_t b = (t & 0x80008000u) | ((t >> 4) & 0x07F007F0u);
      const __nv_bfloat162 r = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&b),
                                       *reinterpret_cast<const __nv_bfloat162*>(&factor));
      out[i] = *reinterpret_cast<const uint32_t*>(&r);
    } else {
      const uint32_t b = (t & 0x80008000u) | ((t >> 1) & 0x3F803F80u);
      const __half2 r = __hmul2(*reinterpret_cast<const __half2*>(&b),
                                *reinterpret_cast<const __half2*>(&factor));
      out[i] = *reinterpret_cast<const uint32_t*>(&r);
    }
  }
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

// DT: 0 = fp16, 1 = bf16 (dY and dW).  SPLIT: partial sums to the workspace (tmC is then the
// workspace's map).  DEBUG adds fault injection.
template <int DT, bool SPLIT, bool DEBUG>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kWgThreads, 1)
    wgrad_pair_kernel(const __grid_constant__ CUtensorMap tmQ,
                      const __grid_constant__ CUtensorMap tmB,
                      const __grid_constant__ CUtensorMap tmC, const WgradParams p) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ WgradCtl ctl;

  const uint32_t warp = threadIdx.x >> 5;
  const uint32_t lane = threadIdx.x & 31u;
  const uint32_t rank = cluster_ctarank();
  const uint32_t pair = blockIdx.x >> 1;
  const uint32_t num_pairs = gridDim.x >> 1;
  const uint32_t sbase = (smem_u32(smem_raw) + 1023u) & ~1023u;
  const uint32_t sA0 = sbase;                      // stage s: A, then B, then the raw bytes
  const uint32_t sB0 = sA0 + kWgABytes;
  const uint32_t sR0 = sB0 + kWgBBytes;
  const uint32_t sEpi = sbase + kWgStages * kWgStageBytes;

  const uint32_t bar_loaded = smem_u32(&ctl.loaded[0]);
  const uint32_t bar_made = smem_u32(&ctl.made[0]);
  const uint32_t bar_raw = smem_u32(&ctl.raw[0]);
  const uint32_t bar_consumed = smem_u32(&ctl.consumed[0]);
  const uint32_t bar_tmem_full = smem_u32(&ctl.tmem_full[0]);
  const uint32_t bar_tmem_empty = smem_u32(&ctl.tmem_empty[0]);
  const uint32_t bar_drain = smem_u32(&ctl.drain);

  if (threadIdx.x == 0) {
#pragma unroll
    for (int s = 0; s < kWgStages; ++s) {
      mbar_init(bar_loaded + 8u * s, 1);
      mbar_init(bar_made + 8u * s, kWgMakeWarps);
      mbar_init(bar_raw + 8u * s, 1);
      mbar_init(bar_consumed + 8u * s, 1);
      ctl.fills.par[s] = 0;
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
    // ------------------------------------------------------------ TMA producer (both CTAs)
    if (lane == 0) {
      uint32_t pending = 0, pending_par = 0;   // raw fills that may still be in flight
      bool ok = true;
      uint64_t phase = 0;
      for (WgradUnits un(p, pair, num_pairs); ok && un.valid(); un.next()) {
        const PersistentTileScheduler& sched = un.sched;
        const bool half = sched.half_unit();
        const int32_t m0 = static_cast<int32_t>(sched.m_idx * kPairBM + rank * kBM);
        const int32_t n0 = static_cast<int32_t>(sched.n_idx * kBN) +
                           (half ? sched.part * (kBN / 2) +
                                       static_cast<int32_t>(rank) * (kPairBNHalf / 2)
                                 : static_cast<int32_t>(rank) * kPairBNHalf);
        const uint32_t b_chunks = half ? 1u : 2u;
        const uint32_t tx_bytes = 2u * b_chunks * kWgChunkBytes;
        for (uint32_t k = un.k_lo; k < un.k_hi; ++k, ++phase) {
          const uint32_t s = static_cast<uint32_t>(phase % kWgStages);
          const uint32_t par = static_cast<uint32_t>((phase / kWgStages) & 1u);
          if (!pair_wait_or_abort(bar_consumed + 8u * s, par ^ 1u, abort_flag, peer_abort, limit,
                                  kRoleProducer)) {
            ok = false;
            break;
          }
          pending &= ~(1u << s);   // its bytes were turned and multiplied
          if (DEBUG && injected_skip(p.inject_skip_phase, phase))
            continue;  // injected fault: this CTA never arms or fills this phase
          const int32_t kx = static_cast<int32_t>(k) * kWgBK;
          mbar_arrive_expect_tx(bar_raw + 8u * s, kWgRawBytes);
          tma_load_2d(sR0 + s * kWgStageBytes, &tmQ, bar_raw + 8u * s, m0, kx);
          pending |= 1u << s;
          pending_par = (pending_par & ~(1u << s)) | (par << s);
          const uint32_t full_even = mapa_shared(bar_loaded + 8u * s, 0);
          if (rank == 0) mbar_arrive_expect_tx(bar_loaded + 8u * s, tx_bytes);
#pragma unroll
          for (uint32_t c = 0; c < 2; ++c) {
            if (c >= b_chunks) break;
            tma_load_2d_pair(sB0 + s * kWgStageBytes + c * kWgChunkBytes, &tmB, full_even,
                             n0 + static_cast<int32_t>(c * kBChunkCols), kx);
          }
          record_fill(ctl.fills, s, phase, par, tx_bytes / 2u);
        }
      }
      if (!ok) {
        for (uint32_t s = 0; s < kWgStages; ++s)
          if ((pending >> s) & 1u)
            wait_bounded(bar_raw + 8u * s, (pending_par >> s) & 1u, limit, kRoleDrain);
      }
      // the odd producer has stopped filling: its records are final (see pair_drain_fills)
      if (rank == 1) mbar_arrive_cluster(mapa_shared(smem_u32(&ctl.odd_done), 0));
    }
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer (even CTA)
    if (lane == 0 && rank == 0) {
      constexpr uint32_t idesc_full = idesc_f16(DT, kPairBM, kBN, /*A M-major*/ 1, /*B N-major*/ 1);
      constexpr uint32_t idesc_half = idesc_f16(DT, kPairBM, kBN / 2, 1, 1);
      bool ok = true;
      uint64_t phase = 0;
      for (WgradUnits un(p, pair, num_pairs); ok && un.valid(); un.next()) {
        const uint32_t w = un.w;
        const uint32_t buf = w & 1u;
        if (!pair_wait_or_abort<true>(bar_tmem_empty + 8u * buf, ((w >> 1) & 1u) ^ 1u, abort_flag,
                                      peer_abort, limit, kRoleMma)) {
          ok = false;
          break;
        }
        tcgen05_fence_after_sync();
        const uint32_t d_tmem = tmem_base + buf * kBN;
        const uint32_t idesc = un.sched.half_unit() ? idesc_half : idesc_full;
        for (uint32_t k = un.k_lo; k < un.k_hi; ++k, ++phase) {
          const uint32_t s = static_cast<uint32_t>(phase % kWgStages);
          const uint32_t par = static_cast<uint32_t>((phase / kWgStages) & 1u);
          if (!pair_wait_or_abort(bar_loaded + 8u * s, par, abort_flag, peer_abort, limit,
                                  kRoleMma) ||
              !pair_wait_or_abort<true>(bar_made + 8u * s, par, abort_flag, peer_abort, limit,
                                        kRoleMma)) {
            ok = false;
            break;
          }
          tcgen05_fence_after_sync();
#pragma unroll
          for (uint32_t kk = 0; kk < kWgBK / kUmmaK; ++kk) {
            // both operands: 16 tokens = 2048 bytes on; LBO = the next 64 columns
            const uint32_t off = s * kWgStageBytes + kk * kUmmaK * 128u;
            const uint64_t a_desc = smem_desc_sw128(sA0 + off, kWgChunkBytes, 1024);
            const uint64_t b_desc = smem_desc_sw128(sB0 + off, kWgChunkBytes, 1024);
            umma_f16_pair(d_tmem, a_desc, b_desc, idesc, (k != un.k_lo || kk != 0u) ? 1u : 0u);
          }
          umma_commit_pair_multicast(bar_consumed + 8u * s, 0x3);
        }
        if (!ok) break;
        umma_commit_pair_multicast(bar_tmem_full + 8u * buf, 0x3);
      }
      umma_commit_pair_multicast(bar_drain, 0x1);
      wait_bounded(bar_drain, 0, limit, kRoleDrain);
    }
    __syncwarp();
  } else if (warp >= kWgFirstMakeWarp) {
    // ------------------------------------------------------------ checkpoint bytes -> A operand
    // Eight threads take a token's 128 bytes, 16 each; the warps' threads cover 16 tokens at a
    // time.  A warp reads 512 neighbouring bytes; a thread writes its 32 bytes as two 16-byte
    // chunks of the token's row of column chunk c / 4, and the threads of column chunk 1 write
    // their second one first, so that eight threads never meet in a bank.
    const uint32_t tt = threadIdx.x - kWgFirstMakeWarp * 32u;
    const uint32_t c = tt & 7u, r0 = tt >> 3;
    const uint32_t sink_even = mapa_shared(smem_u32(&ctl.sink[warp - kFirstEpiWarp]), 0);
    uint64_t phase = 0;
    bool ok = true;
    for (WgradUnits un(p, pair, num_pairs); ok && un.valid(); un.next()) {
      const uint32_t m0 = un.sched.m_idx * kPairBM + rank * kBM;
      const uint32_t sc = m0 / kCkptBlock + c / 2u;     // this thread's scale column
      const bool sc_in = sc < p.scale_cols;
      uint32_t next_s[kWgPasses];
      auto fetch_scales = [&](uint32_t k) {             // zero bytes lie past the ends: any scale
#pragma unroll
        for (uint32_t i = 0; i < kWgPasses; ++i) {
          const uint32_t t = k * kWgBK + i * 16u + r0;
          next_s[i] = sc_in && k < un.k_hi && t < p.K
                          ? p.scales[static_cast<uint64_t>(t) * p.scale_cols + sc]
                          : 127u;
        }
      };
      fetch_scales(un.k_lo);
      for (uint32_t k = un.k_lo; k < un.k_hi; ++k, ++phase) {
        const uint32_t s = static_cast<uint32_t>(phase % kWgStages);
        const uint32_t par = static_cast<uint32_t>((phase / kWgStages) & 1u);
        uint32_t scale[kWgPasses];
#pragma unroll
        for (uint32_t i = 0; i < kWgPasses; ++i) scale[i] = next_s[i];
        fetch_scales(k + 1);
        const bool got = pair_wait_or_abort(bar_raw + 8u * s, par, abort_flag, peer_abort, limit,
                                            kRoleProducer);
        if (!__all_sync(0xffffffffu, got)) {
          ok = false;
          break;
        }
        const uint32_t raw = sR0 + s * kWgStageBytes, a = sA0 + s * kWgStageBytes;
#pragma unroll
        for (uint32_t i = 0; i < kWgPasses; ++i) {
          const uint32_t r = i * 16u + r0;
          uint32_t in[4], out[8];
          ld_shared_v4(raw + r * 128u + c * 16u, in[0], in[1], in[2], in[3]);
          widen16<DT>(in, scale[i], out);
          const uint32_t row = a + (c / 4u) * kWgChunkBytes + r * 128u;
          const uint32_t u0 = 2u * (c & 3u);
          const bool swap = c >= 4u;
#pragma unroll
          for (uint32_t h = 0; h < 2; ++h) {
            const uint32_t unit = u0 + (swap ? 1u - h : h);
            const bool second = swap ? h == 0u : h == 1u;
            st_shared_v4(row + ((unit ^ (r & 7u)) << 4), second ? out[4] : out[0],
                         second ? out[5] : out[1], second ? out[6] : out[2],
                         second ? out[7] : out[3]);
          }
        }
        fence_proxy_async_shared();
        pair_report_warp(bar_made + 8u * s, rank, lane, sink_even);
      }
    }
    __syncwarp();
  } else if (warp >= kFirstEpiWarp) {
    // ------------------------------------------------------------ epilogue (both CTAs)
    const uint32_t q = warp - kFirstEpiWarp;
    const uint32_t sink_even = mapa_shared(smem_u32(&ctl.sink[q]), 0);
    uint32_t chunk = 0;
    for (WgradUnits un(p, pair, num_pairs); un.valid(); un.next()) {
      const uint32_t w = un.w;
      const uint32_t buf = w & 1u;
      const bool got = pair_wait_or_abort(bar_tmem_full + 8u * buf, (w >> 1) & 1u, abort_flag,
                                          peer_abort, limit, kRoleEpilogue);
      if (!__all_sync(0xffffffffu, got)) break;
      tcgen05_fence_after_sync();
      const bool half = un.sched.half_unit();
      const int32_t row0 =
          static_cast<int32_t>(un.sched.m_idx * kPairBM + rank * kBM + q * 32u);
      const int32_t col0 = static_cast<int32_t>(un.sched.n_idx) * kBN +
                           (half ? un.sched.part * (kBN / 2) : 0);
      const uint32_t chunks = half ? kBN / kEpiN / 2 : kBN / kEpiN;
      const uint32_t t_row = tmem_base + ((q * 32u) << 16) + buf * kBN;
#pragma unroll 1
      for (uint32_t j = 0; j < chunks; ++j, ++chunk) {
        uint32_t v[64];
        tmem_ld_32x32b_x64(t_row + j * kEpiN, v);
        if (j == chunks - 1) {
          tcgen05_fence_before_sync();
          pair_report_warp(bar_tmem_empty + 8u * buf, rank, lane, sink_even);
        }
        const int32_t x = col0 + static_cast<int32_t>(j * kEpiN);
        if constexpr (SPLIT) {
          wgrad_store_partial(v, lane, sEpi + q * 2u * kEpiBufBytes, &tmC,
                              static_cast<int32_t>(un.split * p.m_blocks * kPairBM) + row0, x,
                              p.N);
        } else {
          epilogue_store_chunk<DT>(v, lane, sEpi + (q * 2u + (chunk & 1u)) * kEpiBufBytes, &tmC, p,
                                   row0, x);
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

// dW = the sum of the splits' partial sums [splits][part_rows][outs], rounded once.  A thread takes
// 8 neighbouring columns of a row (outs is a multiple of 8).
template <int DT>
__global__ void __launch_bounds__(256)
    wgrad_join_kernel(const float* __restrict__ partials, uint32_t splits, uint64_t split_stride,
                      uint32_t rows, uint32_t outs, void* __restrict__ dw, int64_t ld_dw) {
  grid_dependency_wait();
  grid_launch_dependents();
  const uint32_t vecs = outs / 8u;
  const uint64_t total = static_cast<uint64_t>(rows) * vecs;
  for (uint64_t i = static_cast<uint64_t>(blockIdx.x) * blockDim.x + threadIdx.x; i < total;
       i += static_cast<uint64_t>(gridDim.x) * blockDim.x) {
    const uint32_t row = static_cast<uint32_t>(i / vecs), v = static_cast<uint32_t>(i % vecs);
    const float4* src = reinterpret_cast<const float4*>(partials + static_cast<uint64_t>(row) * outs) + 2u * v;
    float4 a = src[0], b = src[1];
    for (uint32_t s = 1; s < splits; ++s) {
      src += split_stride / 4u;
      const float4 c = src[0], d = src[1];
      a.x += c.x; a.y += c.y; a.z += c.z; a.w += c.w;
      b.x += d.x; b.y += d.y; b.z += d.z; b.w += d.w;
    }
    uint4 o;
    o.x = pack_out<DT>(__float_as_uint(a.x), __float_as_uint(a.y));
    o.y = pack_out<DT>(__float_as_uint(a.z), __float_as_uint(a.w));
    o.z = pack_out<DT>(__float_as_uint(b.x), __float_as_uint(b.y));
    o.w = pack_out<DT>(__float_as_uint(b.z), __float_as_uint(b.w));
    *reinterpret_cast<uint4*>(static_cast<char*>(dw) +
                              (static_cast<int64_t>(row) * ld_dw + 8 * v) * 2) = o;
  }
}

}  // namespace tg
