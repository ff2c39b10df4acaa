// tg_wgrad_config.h -- compile-time constants of the weight-gradient kernel (tg_wgrad_kernel.cuh),
// shared by that kernel and the host code that sizes its launch and tensor maps.
#pragma once

#include "tg_config.h"

namespace tg {

// Per CTA and k-block of 64 tokens: the A operand, 64 tokens x 128 columns as two chunks of 64
// columns (16 KiB), its half of the dY columns (16 KiB), and the checkpoint bytes the operand is
// made from (8 KiB); four stages.
constexpr int kWgBK = 64;
constexpr int kWgStages = 4;
constexpr uint32_t kWgChunkBytes = kWgBK * kBChunkCols * kElemBytes;   // 8 KiB: 64 x 64 values
constexpr uint32_t kWgABytes = 2 * kWgChunkBytes;
constexpr uint32_t kWgBBytes = 2 * kWgChunkBytes;
constexpr uint32_t kWgRawBytes = kWgBK * kBM;
constexpr uint32_t kWgStageBytes = kWgABytes + kWgBBytes + kWgRawBytes;   // 40 KiB
constexpr uint32_t kWgSmemBytes = kSmemAlignSlack + kWgStages * kWgStageBytes + kEpiSmemBytes;
// warps 0..7 as in the GEMM; warps 8..11 make the A operand
constexpr int kWgFirstMakeWarp = 8;
constexpr int kWgMakeWarps = 4;
constexpr int kWgThreads = 32 * (kWgFirstMakeWarp + kWgMakeWarps);
constexpr uint32_t kWgPasses = kWgBK * kBM / (16 * 32 * kWgMakeWarps);   // 16 bytes a thread each
static_assert(kWgSmemBytes + 512 <= 232448, "shared memory per CTA (weight gradient)");
static_assert(kWgStageBytes % 1024 == 0 && kWgChunkBytes % 1024 == 0, "swizzle atoms aligned");

}  // namespace tg
