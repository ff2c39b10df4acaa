// Host build of the walk over the fused products' units (tg_linear_units.h, compiled with the CUDA qualifiers
// defined away) for the CPU tests: random launches of one or two products, in which the workers together take
// every tile's every range of K once.
// usage: linear_units_driver seed launches.  Prints "ok two ahead halves splits" (how often) or what is wrong.
#include <cstdio>
#include <cstdlib>
#include <random>
#include <vector>

#include "tg_linear_units.h"

namespace {

std::mt19937 rng;
uint32_t upto(uint32_t n) { return 1 + rng() % n; }

[[noreturn]] void wrong(const char* what) {
  printf("wrong: %s\n", what);
  exit(1);
}

tg::LinearProblem product(uint32_t pairs) {
  tg::LinearProblem q = {};
  q.m_blocks = upto(12);
  q.n_blocks = upto(12);
  q.k_blocks = upto(40);
  q.group = upto(12);
  q.column_major = rng() % 2;
  const uint32_t tiles = q.m_blocks * q.n_blocks;
  q.split_from = q.total_units = tiles;
  q.splits = 1;
  q.blocks_per_split = q.k_blocks;
  if (rng() % 2) {
    q.blocks_per_split = upto(q.k_blocks);
    q.splits = (q.k_blocks + q.blocks_per_split - 1) / q.blocks_per_split;
  } else if (rng() % 2) {
    tg::PersistentTileScheduler::tail_split(tiles, pairs, q.split_from, q.total_units);
  }
  return q;
}

// Every tile's k-blocks, by halves, taken so far.
template <int PRODUCTS>
void launch(const tg::LinearWalk& w, uint32_t workers) {
  std::vector<std::vector<int>> taken(2);
  for (int i = 0; i < PRODUCTS; ++i) taken[i].resize(w.q[i].m_blocks * w.q[i].n_blocks * w.q[i].k_blocks * 2);
  for (uint32_t c = 0; c < workers; ++c)
    for (tg::LinearUnits<PRODUCTS> un(w, c, workers); un.valid(); un.next()) {
      const tg::LinearProblem& q = un.q();
      if (un.sched.m_idx >= q.m_blocks || un.sched.n_idx >= q.n_blocks) wrong("a tile that is not there");
      if (un.k_lo >= un.k_hi || un.k_hi > q.k_blocks) wrong("k-blocks that are not there");
      for (uint32_t k = un.k_lo; k < un.k_hi; ++k)
        for (int half = 0; half < 2; ++half)
          if (!un.sched.half_unit() || un.sched.part == half)
            ++taken[un.product()][((un.sched.m_idx * q.n_blocks + un.sched.n_idx) * q.k_blocks + k) * 2 + half];
    }
  for (const auto& product : taken)
    for (const int n : product)
      if (n != 1) wrong(n ? "a unit is taken twice" : "a unit is left out");
}

}  // namespace

int main(int argc, char** argv) {
  if (argc != 3) return 2;
  rng.seed(std::atoi(argv[1]));
  long two = 0, ahead = 0, halves = 0, splits = 0;
  for (int i = std::atoi(argv[2]); i > 0; --i) {
    const uint32_t pairs = upto(80);
    tg::LinearWalk w = {};
    const int products = 1 + rng() % 2;
    for (int n = 0; n < products; ++n) {
      w.q[n] = product(pairs);
      w.units[n] = w.q[n].total_units * w.q[n].splits;
      halves += w.q[n].split_from != w.q[n].total_units;
      splits += w.q[n].splits > 1;
    }
    const uint32_t all = w.units[0] + w.units[1], workers = all < pairs ? all : pairs;
    if (products == 1) {
      launch<1>(w, workers);
      continue;
    }
    ++two;
    // no more ahead than there is: what the idle workers of the first one's last round take
    const uint32_t idle = workers - w.units[0] % workers;
    if (idle < workers && rng() % 4) {
      const uint32_t share = (w.units[1] + idle - 1) / idle;
      w.extra = rng() % (share + 1);
      ahead += w.extra > 0;
    }
    launch<2>(w, workers);
  }
  printf("ok %ld %ld %ld %ld\n", two, ahead, halves, splits);
  return 0;
}
