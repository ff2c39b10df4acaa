// tg_linear_config.h -- compile-time constants of the products with fused epilogues
// (tg_linear_kernel.cuh), shared by that kernel and the host code that sizes its launches and tensor
// maps.
#pragma once

#include "tg_config.h"

namespace tg {

// What the epilogue does with the accumulator.
enum LinearEpi {
  kEpiStore = 0,    // rounds and stores it, or stores / adds fp32 partial sums
  kEpiGated = 1,    // act(g) u of two products side by side
  kEpiStats = 2,    // maximum and sum of exponentials of each row, and the target's logit
  kEpiDlogits = 3   // (exp(logit - lse) - [column is the target]) weight
};

// A CTA pair's tile is 256 x 256 accumulator columns; two accumulators take turns.  A stage of the ring
// holds two 64-deep K atoms (eight MMAs), 64 KiB per CTA.
//
// The tensor core truncates as it adds, so a long sum falls short by about 2^-25 of itself for every
// step of 16 products: an lse over 4096 columns was 1.6e-6 off, an fp16 gradient summed over a
// vocabulary 1e-3.  So a sum is cut into segments of a few k-blocks, each in an accumulator of its
// own, which the epilogue adds in registers, rounding to nearest.  1024 products of a result that is
// rounded to 16 bits; 512 of a logit, whose statistics stay in fp32.  Measured with 1024 / 512 / 256: lse of
// 2048 x 8192 (fp16, 20000 words) 5.1e-7 / 2.6e-7 / 1.4e-7 off, 381 / 382 / 397 us; 300 x 4096 (bf16,
// 32000 words) 4.0e-7 / 1.9e-7 / 1.0e-7, 90.3 / 90.1 / 94.4 us; products of one sign lose more (512: 1.5e-6 in
// fp16, 5e-7 in bf16).  The backward pass cuts logits alike, so that it makes the forward pass's again bit for
// bit and what they lack cancels in exp(l - lse): of fp16 rows with p = 1 - 2^-11 the target's gradient was 13 %
// off with 1024, now 0.3 %.
constexpr int kLinAtoms = 2;
constexpr int kLinBK = kLinAtoms * kKAtom;                              // 128
constexpr int kLinStages = 3;
// k-blocks of a segment, as a power of two: 1024 products, 512
constexpr uint32_t kLinSegmentLog = 3u, kLogitSegmentLog = 2u;
constexpr uint32_t kLinOperandBytes = kBM * kLinBK * kElemBytes;        // 128 rows or columns: 32 KiB
constexpr uint32_t kLinStageBytes = 2 * kLinOperandBytes;
// warps 0..3 as in the GEMM; eight epilogue warps: warp 4 + e has TMEM lanes 32 (e % 4) .. and half
// e / 4 of the columns, and one staging buffer
constexpr int kLinEpiWarps = 8;
constexpr uint32_t kLinThreads = 32 * (kFirstEpiWarp + kLinEpiWarps);
constexpr uint32_t kLinSmemBytes =
    kSmemAlignSlack + kLinStages * kLinStageBytes + kLinEpiWarps * kEpiBufBytes;
// Registers a thread: an epilogue thread holds 128 sums.  Launched with 168 (384 threads), of which the
// first warpgroup gives back all but 64.
constexpr int kLinLaunchRegs = 168, kLinFewRegs = 64, kLinEpiRegs = 216;
static_assert(kLinSmemBytes + 512 <= 232448, "shared memory per CTA (products)");
static_assert(128 * kLinFewRegs + 256 * kLinEpiRegs <= int(kLinThreads) * kLinLaunchRegs,
              "registers handed over come from the launch's own");

// Columns of a gated product in one tile: half of the accumulator's are g, half u.
constexpr int kGatedTileN = kBN / 2;

// Blocks at most of the pass that makes dg and du of a gated product's gradient (8 an SM): in fp16 each
// leaves its largest value.
constexpr uint32_t kGradBlocks = 2048;

// Rows of one split's partial sums: whole boxes of 32 rows
constexpr uint32_t kPartialRows = 32;

// Statistics of a row: one slot per 64 logits; an epilogue warp has two slots' columns, or one of a half
// unit's
constexpr uint32_t kStatCols = kEpiN;

}  // namespace tg
