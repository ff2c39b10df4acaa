// tg_few_config.h -- compile-time constants of the products with few rows (tg_few_kernel.cuh), shared
// by that kernel and the host code that sizes its launches and tensor maps.
#pragma once

#include "tg_config.h"
#include "tg_linear_config.h"

namespace tg {

constexpr int kFewRows = 64;             // rows at most
// Rows up to which gradients that are rounded on the way come in two terms (past 8 rows of at least 128
// values their errors average out), and up to which gradients towards weights are tg_outer_kernel.cuh's:
// measured (bf16, us, gated backward 1200 x 5896 / 2232 x 2592): 8 rows 22.9 / 20.4, 17 rows on the tensor
// core 24.2 / 20.9, 16 rows without it 38 / 35.
constexpr int kTwoTermRows = 8;
constexpr int kFewM = 128;               // weights' rows or columns (results) in a tile
constexpr int kFewBK = kKAtom;           // 64 of K in a stage
// A sum is cut into segments, as tg_linear_config.h explains: of 1024 products, of logits 128.  Where a
// single row's target is nearly certain its gradient is what 1 - p leaves, and a logit's error counts
// 1 / (1 - p) times (one fp16 row, p = 0.998: gradients 6.1e-4 off with 1024, plain fp32 2.5e-4).
template <int EPI>
constexpr uint32_t kFewSegment = EPI == kEpiStats || EPI == kEpiDlogits ? 2u : 16u;
// Logits of up to 32 rows: an accumulator still has 64 columns, which are 2 or 4 (16 rows) parts that the
// steps of 16 products take turns with, so a part is added to 3 times or once before it is read out.
template <int EPI>
constexpr bool kFewParted = EPI == kEpiStats || EPI == kEpiDlogits;
// warp 0 loads, warp 1 issues the MMAs and owns the TMEM, warps 2..5 are the epilogue
constexpr uint32_t kFewThreads = 192;
constexpr int kFewEpiThreads = 128;
constexpr int kFewMaxCluster = 8;
constexpr int kFewMaxStages = 6;
// Two CTAs share an SM, so that one's start and end fall into the other's loads.
constexpr uint32_t kFewRingBudget = 110u * 1024u;

constexpr uint32_t kFewWeightBytes = kFewM * kFewBK * kElemBytes;       // 16 KiB

// rows as the MMA takes them: 16, 32 or 64
constexpr uint32_t few_padded(int64_t rows) { return rows <= 16 ? 16u : rows <= 32 ? 32u : 64u; }

// n: padded rows, times two where they come in two terms
constexpr uint32_t few_stage_bytes(bool gated, uint32_t n) {
  return (gated ? 2u : 1u) * kFewWeightBytes + n * kFewBK * kElemBytes;
}
constexpr uint32_t few_stages(bool gated, uint32_t n) {
  const uint32_t most = kFewRingBudget / few_stage_bytes(gated, n);
  return most < kFewMaxStages ? most : kFewMaxStages;
}
// the ring, which the sums of a cluster's CTAs take over at the end: 128 x n floats of each product
constexpr uint32_t few_smem_bytes(bool gated, uint32_t n) {
  return kSmemAlignSlack + few_stages(gated, n) * few_stage_bytes(gated, n);
}
static_assert(few_stages(true, 64) >= 2 && few_stages(false, 128) >= 3, "a ring has to run ahead");
// ... or, for statistics, the sums, half as many again by rows (padded) and a pair for each thread
static_assert(2u * kFewM * 64u * 4u <= few_stages(true, 64) * few_stage_bytes(true, 64) &&
              (kFewM * 64u + (kFewM + 1u) * 64u + 2u * 128u + 2u) * 4u <=
                  few_stages(false, 64) * few_stage_bytes(false, 64),
              "sums fit into the ring");

}  // namespace tg
