// tg_wgrad_config.h -- compile-time constants of the weight-gradient kernel (tg_wgrad_kernel.cuh),
// shared by that kernel and the host code that sizes its launch and tensor maps.
#pragma once

#include "tg_config.h"

namespace tg {

// Per CTA and k-block of 64 tokens: the A operand, 64 tokens x 128 columns as two chunks of 64
// columns (16 KiB), and the CTA's half of each 256-column N-half of dY (16 KiB each).  The
// checkpoint bytes A is made from (8 KiB) go through a ring of their own.
constexpr int kWgBK = 64;
constexpr uint32_t kWgChunkBytes = kWgBK * kBChunkCols * kElemBytes;   // 8 KiB: 64 x 64 values
constexpr uint32_t kWgABytes = 2 * kWgChunkBytes;
constexpr uint32_t kWgRawBytes = kWgBK * kBM;
constexpr uint32_t kWgScalePitch = 16;          // a token's 4 scales lie within 16 bytes
constexpr uint32_t kWgScaleBytes = kWgBK * kWgScalePitch;
// warps 0..7 as in the GEMM, but warps 2 and 3 load scales and checkpoint bytes; warps 8.. make the
// A operand, in groups of four that take k-blocks in turn
constexpr int kWgFirstMakeWarp = 8;
constexpr int kWgMakeWarps = 4;   // of one group
constexpr uint32_t kWgPasses = kWgBK * kBM / (16 * 32 * kWgMakeWarps);   // 16 bytes a thread each

// NH: N-halves of 256 columns in a tile.
//
// A group visits a ring slot once in a while only, so a wait by parity must never find the slot two
// turns behind.  Checkpoint ring: with raws % groups == 0 the slot's last turn was the group's own.
// Operand ring: the group's k-block before this one (groups back) was multiplied into a slot that
// k-block p - groups - stages had left, so with groups <= stages k-block p - 2 stages has left too.
template <int NH>
struct WgradConfig {
  static constexpr int kStages = NH == 1 ? 4 : 3;
  static constexpr int kGroups = 2;
  static constexpr int kRaws = 4;
  static constexpr uint32_t kThreads = 32 * (kWgFirstMakeWarp + kGroups * kWgMakeWarps);
  static constexpr uint32_t kBBytes = NH * 2 * kWgChunkBytes;
  static constexpr uint32_t kStageBytes = kWgABytes + kBBytes;   // 32 or 48 KiB
  static constexpr uint32_t kSmemBytes = kSmemAlignSlack + kStages * kStageBytes +
                                         kRaws * (kWgRawBytes + kWgScaleBytes) + kEpiSmemBytes;
  static constexpr int kTileN = NH * kBN;
  static_assert(kSmemBytes + 512 <= 232448, "shared memory per CTA (weight gradient)");
  static_assert(kRaws % kGroups == 0 && kGroups <= kStages, "parities of slots (see above)");
};
static_assert(kWgChunkBytes % 1024 == 0, "swizzle atoms aligned");

}  // namespace tg
