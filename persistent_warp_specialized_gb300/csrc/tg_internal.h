// tg_internal.h -- interface between the C-ABI translation units (tg_api.cu, tg_train_api.cu,
// tg_linear_api.cu) and those that hold the kernels (tg_gemm.cu, tg_train.cu).  Not installed, not
// part of the ABI.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>

namespace tg {

struct GemmLaunch {
  CUtensorMap tmA, tmB, tmC;
  void* C;
  uint32_t M, N, K;
  uint32_t m_blocks, n_blocks, k_blocks, group;
  uint32_t split_from, total_units;
  uint32_t column_major;
  uint32_t dynamic;
  uint32_t epi_direct;
  uint32_t grid;
  uint64_t watchdog_ns;
  int32_t* trace;
  int64_t inject_skip_phase;
  uint32_t sk_tiles, sk_epoch, sk_slot_f4;   // stream-K tail (0 tiles: none)
  uint32_t* sk_flags;
  float4* sk_partials;
};

// the block-scaled MXFP8 GEMM (one CTA per 128 x 256 tile, the single variant's schedule)
struct MxLaunch {
  CUtensorMap tmA, tmB, tmC;
  CUtensorMap tmSFA, tmSFB;   // pair variant: the packed scales as rows of 128 words
  const void* SFA;   // packed scale atoms (mx_pack_scales_kernel)
  const void* SFB;
  uint32_t sfa_blocks, sfb_blocks;   // row blocks of 128 per k-block in the packed arrays
  uint32_t M, N, K;
  uint32_t m_blocks, n_blocks, k_blocks, group;
  uint32_t split_from, total_units;
  uint32_t column_major;
  uint32_t grid;
  uint64_t watchdog_ns;
  int32_t* trace;
  int64_t inject_skip_phase;
};

// kernel variants: one CTA per 128 x 256 tile, or a CTA pair (cta_group::2) per 256 x 256 tile
enum Variant { kVariantSingle = 1, kVariantPair = 2, kVariantPairWide = 3 };

// Sets the dynamic shared-memory limit of every GEMM instantiation on the current device and
// returns how many CTA pairs of the pair kernels can be resident at once (*max_pairs: the
// smaller of the dense and the MXFP8 pair kernel).
cudaError_t prepare_gemm_kernels(int* max_pairs);
// dtype 0 = fp16, 1 = bf16.  For the pair variants l.grid counts CTAs (even) and l.m_blocks
// counts 256-row pair tiles (l.n_blocks: 512-column tiles for kVariantPairWide).
cudaError_t launch_gemm(int dtype, bool debug, int variant, const GemmLaunch& l,
                        cudaStream_t stream);
// out_dtype 0 = fp16, 1 = bf16; variant kVariantSingle or kVariantPair (l.grid counts CTAs)
cudaError_t launch_mxfp8(int out_dtype, bool debug, int variant, const MxLaunch& l,
                         cudaStream_t stream);
// row-major scales [rows, 4 * k_blocks] -> atoms [k_blocks][row_blocks][512]
cudaError_t launch_mx_pack(const void* sf, void* out, uint32_t rows, uint32_t k_blocks,
                           uint32_t row_blocks, cudaStream_t stream);
// C[0 .. bytes) = 0 (bytes a multiple of 16, C 16-byte aligned)
cudaError_t launch_zero_fill(void* C, uint64_t bytes, cudaStream_t stream);
// rows of 5 int32 (worker, w, bx, by, part) over the units [0, units); tiles below
// split_from are whole (part -1)
cudaError_t launch_tile_schedule(uint32_t m_blocks, uint32_t n_blocks, uint32_t num_workers,
                                 uint32_t group, uint32_t split_from, uint32_t units,
                                 uint32_t column_major, int32_t* out_dev, cudaStream_t stream);

// ---------------------------------------------------------------- training operators
// Layer norm of x [rows, cols] (tg_norm_kernel.cuh).  dtype, param_dtype: TG_F16, TG_BF16, TG_F32;
// param_dtype is TG_F32 or dtype.  Null pointers leave out what they stand for.
struct NormLaunch {
  const void *x, *gamma, *beta;
  void* y;
  float *mean, *rstd;
  void *q, *s;           // the checkpoint of y, or null
  int64_t rows, cols, ld_x, ld_y;
  int dtype, param_dtype;
  float eps;
  int sms;
};
cudaError_t launch_norm_fwd(const NormLaunch& l, cudaStream_t stream);

struct NormBwdLaunch {
  const void *dy, *x, *q, *s, *gamma;   // x, or its checkpoint q and s
  const float *mean, *rstd;
  void *dx, *dgamma, *dbeta;
  float* partials;
  int64_t rows, cols, ld_dy, ld_x, ld_dx;
  int dtype, param_dtype;
  int sms;
};
// Bytes of fp32 partial sums that launch_norm_bwd writes for dgamma and dbeta.
int64_t norm_bwd_workspace(int64_t rows, int64_t cols, int sms);
cudaError_t launch_norm_bwd(const NormBwdLaunch& l, cudaStream_t stream);

// 8-bit checkpoints (tg_ckpt8_kernel.cuh)
cudaError_t launch_ckpt8_pack(const void* x, void* q, void* s, int64_t rows, int64_t cols,
                              int64_t ld_x, int dtype, int sms, cudaStream_t stream);
cudaError_t launch_ckpt8_unpack(const void* q, const void* s, void* out, int64_t rows, int64_t cols,
                                int64_t ld_out, int dtype, int sms, cudaStream_t stream);

// Weight gradient from a checkpoint (tg_wgrad_kernel.cuh): the pair kernel, then, with splits > 1,
// the join of its partial sums.
struct WgradLaunch {
  CUtensorMap tmQ, tmB, tmC;    // tmC: dW, or the workspace when splits > 1
  CUtensorMap tmS;              // the scales, when tma_scales
  uint32_t tma_scales;
  const void* scales;
  void* dw;
  float* partials;
  uint32_t cols, outs, tokens, scale_cols;
  int64_t ld_dw;
  uint32_t m_blocks, n_blocks, k_blocks, group, column_major;
  uint32_t split_from, total_units;   // per split
  uint32_t splits, blocks_per_split;
  uint32_t halves;              // N-halves of 256 columns in a tile: 1 or 2
  uint32_t grid;                // CTAs
  uint64_t watchdog_ns;
  int64_t inject_skip_phase;
  int sms;
};
// Sets the kernels' shared memory limits; *max_pairs: how many of their CTA pairs are resident at once.
cudaError_t prepare_wgrad_kernels(int* max_pairs);
cudaError_t launch_wgrad(int dtype, bool debug, const WgradLaunch& l, cudaStream_t stream);

// Products with fused epilogues (tg_linear_kernel.cuh).  Matrices, tile counts and segments as
// LinearProblem has them.
struct LinearProduct {
  CUtensorMap a[2], b[4], c[3];
  bool a_mn, b_mn;              // the operand lies with m (n) contiguous
  uint32_t M, N;
  uint32_t m_blocks, n_blocks, k_blocks, n_seg, k_seg, group, column_major;
  uint32_t split_from, total_units, splits, blocks_per_split;   // units: per split
  uint32_t partial, part_rows;
  uint32_t segment_log;         // 2^segment_log k-blocks share an accumulator
  const float* alpha;
};
// The cross entropy's rows (RowWeights)
struct XentRows {
  const float* dloss;
  const int64_t* targets;
  int64_t ignore;
  uint32_t vocab;
  float* alpha;
};
struct LinearLaunch {
  LinearProduct q[2];
  int products;                 // 1; with kEpiStore also 2, the one with the longer units first
  uint32_t extra;               // units of the second that take as long as one of the first
  int dtype;
  int epi;                      // LinearEpi
  uint32_t act, keep;
  uint32_t first_col, slots;
  void* stats;
  float* hit;
  const float* lse;
  XentRows loss;
  uint32_t grid;                // CTAs
  uint64_t watchdog_ns;
  int64_t inject_skip_phase;
};
// Sets the kernels' shared memory limits; *max_pairs: how many of their CTA pairs are resident at once.
cudaError_t prepare_linear_kernels(int* max_pairs);
cudaError_t launch_linear(const LinearLaunch& l, cudaStream_t stream);

// The same products for few rows (tg_few_kernel.cuh): ``ranks`` CTAs share a tile of 128 results a row,
// and ``groups`` of them cut K, with fp32 sums [groups][rows][outs] where there are several.
struct FewLaunch {
  CUtensorMap w[2], x[2];       // weights and rows; the second ones along K, or of the gated pair
  CUtensorMap x_rest[2];        // terms == 2: what rounding the rows to 16 bits left
  uint32_t terms;
  int dtype;
  bool w_mn;                    // the weights lie with the results' index contiguous
  int epi;                      // LinearEpi
  uint32_t rows, outs, tiles, ranks, groups;
  float* partials;
  uint32_t k_blocks, k_seg;     // of 64
  const float* alpha;
  uint32_t act;
  void *out, *g, *u;
  void* rest;                   // kEpiDlogits: what rounding ``out`` left, or null
  int64_t ld_out, ld_g, ld_u;
  uint32_t first_col, slots;
  void* stats;
  float* hit;
  const float* lse;
  XentRows loss;
  uint64_t watchdog_ns;
  int64_t inject_skip_phase;
};
cudaError_t launch_few(const FewLaunch& l, cudaStream_t stream);

// out[i] [m, n] = alpha (null: 1) a^T b[i] of at most 8 rows, a [rows, m] and b[i] [rows, n] in one or two
// terms (tg_outer_kernel.cuh); ``results`` of them, 1 or 2.
struct OuterLaunch {
  const void *a, *a_rest, *b[2], *b_rest[2];
  void* out[2];
  int64_t ld_a, ld_b, ld_out[2];
  uint32_t rows, m, n;
  int results;
  const float* alpha;
  int dtype, sms;
};
cudaError_t launch_outer(const OuterLaunch& l, cudaStream_t stream);

// out [rows, cols] = alpha (null: 1) times the sum over splits of partials [splits][part_rows][cols];
// up to three at once
struct LinearJoin {
  const float* partials;
  uint32_t splits, part_rows, rows, cols;
  const float* alpha;
  void* out;
  int64_t ld_out;
};
cudaError_t launch_linear_join(const LinearJoin* joins, int count, int dtype, int sms,
                               cudaStream_t stream);

// h = act(g) u of partial sums of g and u, each [splits][part_rows][outs]; g and u too where given
struct GatedJoin {
  const float *g_parts, *u_parts;
  uint32_t splits, part_rows, rows, outs;
  uint32_t act;
  void *h, *g, *u;
  int64_t ld_h, ld_g, ld_u;
  int dtype, sms;
};
cudaError_t launch_gated_join(const GatedJoin& l, cudaStream_t stream);

// dgu [rows, 2 outs] = (dh u act'(g), dh act(g)), side by side (tg_gated_kernel.cuh); rest: null, or the
// same of what rounding them left.  fp16: both times a power of two, *alpha its inverse; tops: kGradBlocks
// values of scratch.
struct GatedGrad {
  const void *dh, *g, *u;
  void *dgu, *rest;
  float *tops, *alpha;          // bf16: not used
  int64_t rows, outs, ld_dh, ld_g, ld_u;
  uint32_t act;
  int dtype, sms;
};
cudaError_t launch_gated_grad(const GatedGrad& l, cudaStream_t stream);

// Cross entropy (tg_xent_kernel.cuh): loss and lse of each row from its statistics.
struct XentJoin {
  const void* stats;     // float2 [rows][slots]
  const float* hit;
  const int64_t* targets;
  int64_t ignore;
  float *loss, *lse;
  uint32_t rows, slots, vocab;
};
cudaError_t launch_xent_join(const XentJoin& l, cudaStream_t stream);
// The same from fp32 parts of the logits [splits][part_rows][pitch], and the gradients of logits from them.
struct XentParts {
  const float* parts;
  uint32_t splits, part_rows, pitch;
};
struct XentDlogits {
  XentRows loss;
  const float* lse;
  void* out;
  uint32_t rows, cols, first_col, pitch_out;
  int dtype, sms;
};
cudaError_t launch_xent_rows(const XentJoin& l, const XentParts& parts, cudaStream_t stream);
cudaError_t launch_xent_dlogits(const XentDlogits& l, const XentParts& parts, cudaStream_t stream);
cudaError_t clear_watchdog_status(cudaStream_t stream);
// synchronises ``stream``, returns the status word in *out and clears it
cudaError_t read_and_clear_watchdog_status(unsigned int* out, cudaStream_t stream);

}  // namespace tg
