// tg_linear_units.h -- the order in which the CTA pairs of tg_linear_kernel.cuh take the units of a launch's
// products.  Plain integer code: the CPU tests build it for the host, with the qualifiers defined away.
#pragma once

#include <cstdint>

#include "tg_tile_scheduler.cuh"

namespace tg {

struct LinearProblem {
  uint32_t M, N;                     // N: of one segment; m_, n_, k_blocks: of all of them
  uint32_t m_blocks, n_blocks, k_blocks, group, column_major;
  uint32_t split_from, total_units, splits, blocks_per_split;   // units: per split
  uint32_t n_seg, k_seg;             // first tile along N, first k-block, of the second matrices
  uint32_t a_mn, b_mn;               // the operand lies with m (n) contiguous; a_mn: b_mn too
  uint32_t partial;                  // kEpiStore: 0 rounded, 1 fp32 stored, 2 fp32 added to what is there
  uint32_t part_rows;                // rows of one split's partial sums
  uint32_t segment_log;              // kEpiStore: 2^segment_log k-blocks share an accumulator
  const float* alpha;                // kEpiStore: a factor of every result, or null
};

// The products of a launch.
struct LinearWalk {
  LinearProblem q[2];                // the second one's units follow the first one's
  uint32_t units[2];                 // of each (0: no second one)
  uint32_t extra;                    // units of the second that take as long as one of the first
};

// One worker's walk over the units of the products in turn: worker, worker + workers, ... (of a product,
// the tile units of every split in turn).  The first product has the longer units.  Workers that go
// without one in its last round take ``extra`` units each of the second one meanwhile, so that all begin the
// second one's rounds together.
template <int PRODUCTS>
struct LinearUnits {
  const LinearWalk& p;
  uint32_t worker, step, at, which, ahead;   // ahead: units of the second one still to take first
  PersistentTileScheduler sched;
  uint32_t split, k_lo, k_hi;

  __device__ LinearUnits(const LinearWalk& params, uint32_t c, uint32_t workers)
      : p(params), worker(c), step(workers), at(c), which(0), ahead(0), sched(1, 1, 1, 1) {
    if (PRODUCTS == 2 && at >= p.units[0]) second();
    decode();
  }
  __device__ uint32_t product() const { return PRODUCTS == 1 ? 0u : which; }
  __device__ bool valid() const { return at < p.units[product()]; }
  __device__ const LinearProblem& q() const { return p.q[product()]; }
  __device__ void second() {
    const uint32_t busy = p.units[0] % step;   // workers with a unit in the first one's last round
    which = 1;
    if (p.extra != 0u && busy != 0u && worker >= busy) {
      ahead = p.extra;
      at = (worker - busy) * p.extra;
    } else {
      rounds();
    }
  }
  __device__ void rounds() {   // behind what was taken ahead
    const uint32_t busy = p.units[0] % step;
    at = worker + (busy != 0u ? (step - busy) * p.extra : 0u);
  }
  __device__ void next() {
    if (PRODUCTS == 1) {
      at += step;
    } else if (ahead > 1u) {
      --ahead;
      ++at;
    } else if (ahead == 1u) {
      ahead = 0;
      rounds();
    } else {
      at += step;
      if (which == 0u && at >= p.units[0]) second();
    }
    decode();
  }
  __device__ void decode() {
    if (!valid()) return;
    const LinearProblem& o = q();
    split = at / o.total_units;
    sched = PersistentTileScheduler(o.m_blocks, o.n_blocks, o.group, step, o.split_from,
                                    o.total_units, o.column_major);
    sched.jump(at - split * o.total_units, 0);
    k_lo = split * o.blocks_per_split;
    k_hi = k_lo + o.blocks_per_split < o.k_blocks ? k_lo + o.blocks_per_split : o.k_blocks;
  }
};

}  // namespace tg
