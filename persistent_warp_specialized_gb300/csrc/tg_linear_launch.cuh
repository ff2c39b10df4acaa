// tg_linear_launch.cuh -- instantiations and launchers of the products with fused epilogues and of the
// small kernels around them: the gated feed-forward projections, the cross entropy of a vocabulary, and
// the input gradient.  Included by tg_gemm.cu, whose watchdog status word the products share.
#pragma once

#include "tg_few_kernel.cuh"
#include "tg_gated_kernel.cuh"
#include "tg_internal.h"
#include "tg_launch.cuh"
#include "tg_outer_kernel.cuh"
#include "tg_linear_kernel.cuh"
#include "tg_xent_kernel.cuh"

namespace tg {

namespace {

RowWeights row_weights_of(const XentRows& l) {
  RowWeights w;
  w.dloss = l.dloss;
  w.targets = l.targets;
  w.ignore = l.ignore;
  w.vocab = l.vocab;
  w.alpha = l.alpha;
  return w;
}

LinearParams params_of(const LinearLaunch& l) {
  LinearParams p = {};
  for (int i = 0; i < l.products; ++i) {
    const LinearProduct& from = l.q[i];
    LinearProblem& to = p.q[i];
    to.M = from.M;
    to.N = from.N;
    to.m_blocks = from.m_blocks;
    to.n_blocks = from.n_blocks;
    to.k_blocks = from.k_blocks;
    to.group = from.group;
    to.column_major = from.column_major;
    to.split_from = from.split_from;
    to.total_units = from.total_units;
    to.splits = from.splits;
    to.blocks_per_split = from.blocks_per_split;
    to.n_seg = from.n_seg;
    to.k_seg = from.k_seg;
    to.a_mn = from.a_mn;
    to.b_mn = from.b_mn;
    to.partial = from.partial;
    to.part_rows = from.part_rows;
    to.segment_log = from.segment_log;
    to.alpha = from.alpha;
    p.units[i] = to.total_units * to.splits;
  }
  p.extra = l.extra;
  p.act = l.act;
  p.keep = l.keep;
  p.first_col = l.first_col;
  p.slots = l.slots;
  p.stats = static_cast<float2*>(l.stats);
  p.hit = l.hit;
  p.lse = l.lse;
  p.rows = row_weights_of(l.loss);
  p.watchdog_ns = l.watchdog_ns;
  p.inject_skip_phase = l.inject_skip_phase;
  return p;
}

// Calls f with the kernel of an epilogue.
template <int DT, typename F>
cudaError_t with_kernel(int epi, F&& f) {
  if (epi == kEpiStore) return f(linear_pair_kernel<DT, kEpiStore>, std::integral_constant<int, 2>());
  if (epi == kEpiGated) return f(linear_pair_kernel<DT, kEpiGated>, std::integral_constant<int, 1>());
  if (epi == kEpiStats) return f(linear_pair_kernel<DT, kEpiStats>, std::integral_constant<int, 1>());
  return f(linear_pair_kernel<DT, kEpiDlogits>, std::integral_constant<int, 1>());
}

template <int DT>
cudaError_t launch_one(const LinearLaunch& l, cudaStream_t stream) {
  return with_kernel<DT>(l.epi, [&](auto kernel, auto products) {
    constexpr int kMost = decltype(products)::value;
    LinearMaps<kMost> maps;
    for (int q = 0; q < kMost; ++q) {
      const LinearProduct& from = l.q[q < l.products ? q : 0];
      for (int i = 0; i < 2; ++i) maps.a[q][i] = from.a[i];
      for (int i = 0; i < 4; ++i) maps.b[q][i] = from.b[i];
      for (int i = 0; i < 3; ++i) maps.c[q][i] = from.c[i];
    }
    return launch_pdl(kernel, dim3(l.grid), kLinThreads, kLinSmemBytes, stream, maps, params_of(l));
  });
}

// Sets up every kernel of one type; *pairs: the least number resident at once so far.
template <int DT>
cudaError_t prepare_one(int* pairs) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.gridDim = dim3(2, 1, 1);
  cfg.blockDim = dim3(kLinThreads, 1, 1);
  cfg.dynamicSmemBytes = kLinSmemBytes;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  for (int epi = kEpiStore; epi <= kEpiDlogits; ++epi) {
    const cudaError_t e = with_kernel<DT>(epi, [&](auto kernel, auto) {
      cudaError_t err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             static_cast<int>(kLinSmemBytes));
      // a launch with fewer registers could not hand over what its epilogue warps wait for
      cudaFuncAttributes fa;
      if (err == cudaSuccess) err = cudaFuncGetAttributes(&fa, kernel);
      if (err == cudaSuccess && fa.numRegs != kLinLaunchRegs) err = cudaErrorInvalidKernelImage;
      int n = 0;
      if (err == cudaSuccess) err = cudaOccupancyMaxActiveClusters(&n, kernel, &cfg);
      if (err == cudaSuccess && n < *pairs) *pairs = n;
      return err;
    });
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

// As with_kernel, for the products with few rows.
template <int DT, typename F>
cudaError_t with_few_kernel(bool w_mn, int epi, F&& f) {
  if (epi == kEpiGated) return w_mn ? f(few_rows_kernel<DT, 1, kEpiGated>) : cudaErrorInvalidValue;
  if (epi == kEpiStore)
    return w_mn ? f(few_rows_kernel<DT, 1, kEpiStore>) : f(few_rows_kernel<DT, 0, kEpiStore>);
  if (w_mn) return cudaErrorInvalidValue;
  if (epi == kEpiStats) return f(few_rows_kernel<DT, 0, kEpiStats>);
  return f(few_rows_kernel<DT, 0, kEpiDlogits>);
}

template <int DT>
cudaError_t prepare_few() {
  for (int epi = kEpiStore; epi <= kEpiDlogits; ++epi)
    for (int w_mn = 0; w_mn < 2; ++w_mn) {
      if (epi != kEpiStore && w_mn != (epi == kEpiGated)) continue;
      const cudaError_t e = with_few_kernel<DT>(w_mn, epi, [&](auto kernel) {
        uint32_t smem = 0;
        for (uint32_t n = 16; n <= 2 * kFewRows; n *= 2)
          smem = few_smem_bytes(epi == kEpiGated, n) > smem ? few_smem_bytes(epi == kEpiGated, n) : smem;
        const cudaError_t err = cudaFuncSetAttribute(
            kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
        return err != cudaSuccess
                   ? err
                   : cudaFuncSetAttribute(kernel, cudaFuncAttributePreferredSharedMemoryCarveout,
                                          cudaSharedmemCarveoutMaxShared);   // two CTAs an SM
      });
      if (e != cudaSuccess) return e;
    }
  return cudaSuccess;
}

template <int DT>
cudaError_t launch_few_one(const FewLaunch& l, const FewMaps& maps, const FewParams& p,
                           cudaStream_t stream) {
  return with_few_kernel<DT>(l.w_mn, l.epi, [&](auto kernel) {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = l.ranks;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.gridDim = dim3(l.tiles * l.groups * l.ranks);
    cfg.blockDim = dim3(kFewThreads);
    cfg.dynamicSmemBytes = few_smem_bytes(l.epi == kEpiGated, p.n_pad * p.terms);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kernel, maps, p);
  });
}

uint32_t blocks_for(uint64_t threads, int sms, uint32_t most_per_sm) {
  const uint64_t want = (threads + 255) / 256, most = static_cast<uint64_t>(sms) * most_per_sm;
  return static_cast<uint32_t>(want < most ? want : most);
}

}  // namespace

cudaError_t prepare_linear_kernels(int* max_pairs) {
  int pairs = 1 << 20;
  cudaError_t e = prepare_one<0>(&pairs);
  if (e == cudaSuccess) e = prepare_one<1>(&pairs);
  if (e == cudaSuccess) e = prepare_few<0>();
  if (e == cudaSuccess) e = prepare_few<1>();
  *max_pairs = pairs;
  return e;
}

cudaError_t launch_linear(const LinearLaunch& l, cudaStream_t stream) {
  return l.dtype == 0 ? launch_one<0>(l, stream) : launch_one<1>(l, stream);
}

cudaError_t launch_few(const FewLaunch& l, cudaStream_t stream) {
  FewMaps maps;
  FewParams p;
  for (int i = 0; i < 2; ++i) maps.w[i] = l.w[i], maps.x[i] = l.x[i], maps.x_rest[i] = l.x_rest[i];
  p.rows = l.rows;
  p.n_pad = few_padded(l.rows);
  p.outs = l.outs;
  p.k_blocks = l.k_blocks;
  p.k_seg = l.k_seg;
  p.tiles = l.tiles;
  p.groups = l.groups;
  p.partials = l.partials;
  p.terms = l.terms;
  p.stages = few_stages(l.epi == kEpiGated, p.n_pad * p.terms);
  p.stage_bytes = few_stage_bytes(l.epi == kEpiGated, p.n_pad * p.terms);
  p.alpha = l.alpha;
  p.act = l.act;
  p.rest = l.rest;
  p.out = l.out;
  p.g = l.g;
  p.u = l.u;
  p.ld_out = l.ld_out;
  p.ld_g = l.ld_g;
  p.ld_u = l.ld_u;
  p.loss = row_weights_of(l.loss);
  p.first_col = l.first_col;
  p.stats = static_cast<float2*>(l.stats);
  p.slots = l.slots;
  p.hit = l.hit;
  p.lse = l.lse;
  p.watchdog_ns = l.watchdog_ns;
  p.inject_skip_phase = l.inject_skip_phase;
  return l.dtype == 0 ? launch_few_one<0>(l, maps, p, stream)
                      : launch_few_one<1>(l, maps, p, stream);
}

namespace {

template <int DT>
cudaError_t launch_outer_one(const OuterParams& p, dim3 grid, cudaStream_t stream) {
  auto run = [&](auto kernel) { return launch_pdl(kernel, grid, kOuterThreads, 0, stream, p); };
  if (p.rows <= 1) return run(outer_kernel<DT, 1>);
  if (p.rows <= 2) return run(outer_kernel<DT, 2>);
  if (p.rows <= 4) return run(outer_kernel<DT, 4>);
  return run(outer_kernel<DT, 8>);
}

}  // namespace

cudaError_t launch_outer(const OuterLaunch& l, cudaStream_t stream) {
  OuterParams p;
  p.a = l.a;
  p.a_rest = l.a_rest;
  for (int i = 0; i < 2; ++i) {
    p.b[i] = l.b[i];
    p.b_rest[i] = l.b_rest[i];
    p.out[i] = l.out[i];
    p.ld_out[i] = l.ld_out[i];
  }
  p.ld_a = l.ld_a;
  p.ld_b = l.ld_b;
  p.rows = l.rows;
  p.m = l.m;
  p.n = l.n;
  p.alpha = l.alpha;
  // as long a walk down m as leaves four blocks an SM: a block reads its columns of b once
  const uint64_t across = static_cast<uint64_t>((l.n + kOuterCols - 1) / kOuterCols) * l.results;
  p.block_m = kOuterMostM;
  while (p.block_m > 16u && across * ((l.m + p.block_m - 1) / p.block_m) < 4ull * l.sms) p.block_m /= 2;
  // blockIdx.y goes up to 65535: the rows of m that one launch takes
  const uint32_t most = p.block_m * 65535u;
  for (uint32_t m0 = 0; m0 < l.m; m0 += most) {
    OuterParams part = p;
    part.m = l.m - m0 < most ? l.m - m0 : most;
    part.a = static_cast<const char*>(p.a) + 2ull * m0;
    if (p.a_rest != nullptr) part.a_rest = static_cast<const char*>(p.a_rest) + 2ull * m0;
    for (int i = 0; i < l.results; ++i)
      part.out[i] = static_cast<char*>(p.out[i]) + 2ll * m0 * p.ld_out[i];
    const dim3 grid((l.n + kOuterCols - 1) / kOuterCols, (part.m + p.block_m - 1) / p.block_m, l.results);
    const cudaError_t e = l.dtype == 0 ? launch_outer_one<0>(part, grid, stream)
                                       : launch_outer_one<1>(part, grid, stream);
    if (e != cudaSuccess || l.m - m0 <= most) return e;
  }
  return cudaSuccess;
}

cudaError_t launch_linear_join(const LinearJoin* joins, int count, int dtype, int sms,
                               cudaStream_t stream) {
  JoinJobs jobs = {};
  uint32_t blocks = 1;
  for (int i = 0; i < count; ++i) {
    const LinearJoin& l = joins[i];
    JoinParams& p = jobs.job[i];
    p.partials = l.partials;
    p.alpha = l.alpha;
    p.out = l.out;
    p.ld_out = l.ld_out;
    p.stride4 = static_cast<uint64_t>(l.part_rows) * l.cols / 4u;
    p.splits = l.splits;
    p.rows = l.rows;
    p.cols = l.cols;
    const uint32_t want = blocks_for(static_cast<uint64_t>(l.rows) * (l.cols / 4u), sms, 8);
    blocks = want > blocks ? want : blocks;
  }
  const dim3 grid(blocks, count);
  return dtype == 0 ? launch_pdl(linear_join_kernel<0>, grid, 256, 0, stream, jobs)
                    : launch_pdl(linear_join_kernel<1>, grid, 256, 0, stream, jobs);
}

cudaError_t launch_gated_join(const GatedJoin& l, cudaStream_t stream) {
  GatedJoinParams p;
  p.g_parts = l.g_parts;
  p.u_parts = l.u_parts;
  p.split_stride = static_cast<uint64_t>(l.part_rows) * l.outs;
  p.splits = l.splits;
  p.rows = l.rows;
  p.outs = l.outs;
  p.act = l.act;
  p.h = l.h;
  p.g = l.g;
  p.u = l.u;
  p.ld_h = l.ld_h;
  p.ld_g = l.ld_g;
  p.ld_u = l.ld_u;
  const dim3 grid(blocks_for(static_cast<uint64_t>(l.rows) * (l.outs / 4u), l.sms, 8));
  return l.dtype == 0 ? launch_pdl(gated_join_kernel<0>, grid, 256, 0, stream, p)
                      : launch_pdl(gated_join_kernel<1>, grid, 256, 0, stream, p);
}

cudaError_t launch_gated_grad(const GatedGrad& l, cudaStream_t stream) {
  GatedGradParams p;
  p.dh = l.dh;
  p.g = l.g;
  p.u = l.u;
  p.dgu = l.dgu;
  p.rest = l.rest;
  p.ld_dh = l.ld_dh;
  p.ld_g = l.ld_g;
  p.ld_u = l.ld_u;
  p.rows = static_cast<uint32_t>(l.rows);
  p.vecs = static_cast<uint32_t>(l.outs / 8);
  p.act = l.act;
  p.tops = l.tops;
  p.alpha = l.alpha;
  const uint32_t blocks = blocks_for(static_cast<uint64_t>(p.rows) * p.vecs, l.sms, 8);
  const dim3 grid(blocks < kGradBlocks ? blocks : kGradBlocks);
  auto run = [&](auto kernel) { return launch_pdl(kernel, grid, 256, 0, stream, p); };
  const bool two = l.rest != nullptr;
  if (l.dtype != 0)
    return two ? run(gated_grad_kernel<1, true, false>) : run(gated_grad_kernel<1, false, false>);
  const cudaError_t e =
      two ? run(gated_grad_kernel<0, true, false>) : run(gated_grad_kernel<0, false, false>);
  if (e != cudaSuccess) return e;
  return two ? run(gated_grad_kernel<0, true, true>) : run(gated_grad_kernel<0, false, true>);
}

namespace {

XentJoinParams xent_params_of(const XentJoin& l) {
  XentJoinParams p;
  p.stats = static_cast<const float2*>(l.stats);
  p.hit = l.hit;
  p.targets = l.targets;
  p.ignore = l.ignore;
  p.loss = l.loss;
  p.lse = l.lse;
  p.rows = l.rows;
  p.slots = l.slots;
  p.vocab = l.vocab;
  return p;
}

LogitParts parts_of(const XentParts& l) {
  LogitParts p;
  p.parts = l.parts;
  p.stride4 = static_cast<uint64_t>(l.part_rows) * l.pitch / 4u;
  p.splits = l.splits;
  p.pitch4 = l.pitch / 4u;
  return p;
}

}  // namespace

cudaError_t launch_xent_join(const XentJoin& l, cudaStream_t stream) {
  return launch_pdl(xent_join_kernel, dim3((l.rows + 3u) / 4u), 128, 0, stream, xent_params_of(l));
}

cudaError_t launch_xent_rows(const XentJoin& l, const XentParts& parts, cudaStream_t stream) {
  return launch_pdl(xent_rows_kernel, dim3(l.rows), 128, 0, stream, xent_params_of(l),
                    parts_of(parts));
}

cudaError_t launch_xent_dlogits(const XentDlogits& l, const XentParts& parts, cudaStream_t stream) {
  DlogitsParams p;
  p.parts = parts_of(parts);
  p.rows = row_weights_of(l.loss);
  p.lse = l.lse;
  p.out = l.out;
  p.m = l.rows;
  p.n = l.cols;
  p.first_col = l.first_col;
  p.pitch_out = l.pitch_out;
  const dim3 grid(blocks_for(static_cast<uint64_t>(l.rows) * ((l.cols + 3u) / 4u), l.sms, 4));
  return l.dtype == 0 ? launch_pdl(xent_dlogits_kernel<0>, grid, 256, 0, stream, p)
                      : launch_pdl(xent_dlogits_kernel<1>, grid, 256, 0, stream, p);
}

}  // namespace tg
