// tg_linear_api.cu -- the C ABI of the operators between the norm and the loss (include/tg.h): the
// gated feed-forward projections, the cross entropy of a vocabulary projection, a linear layer's input
// gradient.  Argument checks, plans of the products, workspaces and launches.
#include <cuda_runtime.h>

#include <cstdint>
#include <initializer_list>

#include "../../include/tg.h"
#include "tg_api_checks.h"
#include "tg_api_common.h"
#include "tg_few_config.h"
#include "tg_internal.h"
#include "tg_linear_config.h"
#include "tg_tile_scheduler.cuh"

using namespace tg::abi;

namespace {

// A matrix as it lies in memory: ``rows`` rows of ``cols`` values, ``ld`` values apart.
struct Mat {
  const void* p = nullptr;
  int64_t rows = 0, cols = 0, ld = 0;
  const char* name = "";
};

// D[M, N] = A B, before its plan.  Two matrices may stand in an operand's place (tg_linear_kernel.cuh):
// segs_n: N columns each of b[0], b[1] to c[0], c[1]; segs_k: K values each of a[0], b[0 .. 1] and of
// a[1], b[2 .. 3].  a_rest, b_rest: with few rows, what rounding a[i] and b[i] left.
struct Product {
  int epi = tg::kEpiStore;
  int dtype = 0;
  bool a_mn = false, b_mn = false;
  int64_t M = 0, N = 0, K = 0;
  int segs_n = 1, segs_k = 1;
  Mat a[2], b[4], c[3], a_rest[2], b_rest[2];
  bool two_terms = false;
  const float* alpha = nullptr;
  // kEpiStore over several launches: 0 alone, 1 the first, 2 a later one, whose fp32 sums are added to
  // the first's; the caller joins them after the last
  int accumulate = 0;
  uint32_t act = 0, keep = 0;
  bool logits = false;      // sums of logits: shorter segments
  uint32_t first_col = 0, slots = 0;
  void* stats = nullptr;
  float* hit = nullptr;
  const float* lse = nullptr;
  tg::XentRows loss = {};
};

// How a product is cut into units.
struct Plan {
  bool few;                 // the kernel for few rows takes it: splits are its groups
  uint32_t ranks;           // of few rows: CTAs that share a tile
  bool outer;               // tg_outer_kernel.cuh takes it, and nothing below counts
  uint32_t m_tiles, n_tiles, n_seg, k_blocks, k_seg, splits, blocks_per_split;
  uint32_t units;           // tiles
  uint32_t part_rows, part_pitch;   // rows of one split's sums, and values from one to the next
  uint64_t partial_bytes;   // fp32 sums of one N segment (0: results are stored rounded)
};

// Microseconds on GB300 that the choice of splits goes by: a k-block of a tile where few pairs are at work
// and where all are (they share the L2); what a unit adds; the join, and bytes of partial sums a
// microsecond, written and read.
constexpr double kBlockUs = 0.35, kFullBlockUs = 0.66, kUnitUs = 0.4, kJoinUs = 3.0;
constexpr double kWriteBytes = 5e6, kReadBytes = 4e6;
constexpr uint32_t kMinBlocks = 4;   // k-blocks of a unit when K is split

// Few rows: the weights are the MMA's larger operand, and clusters share a tile along K.
bool few_rows(const Product& p, bool sums) {
  return p.M <= tg::kFewRows && !p.a_mn && p.segs_n == 1 && !sums;
}

// The plan with K in about ``splits`` ranges.  sums: results go to partial sums in any case.
Plan plan_of(const Product& p, uint32_t splits, bool sums = false) {
  Plan w;
  w.few = w.outer = false;
  w.ranks = 1;
  w.m_tiles = static_cast<uint32_t>(ceil_div(p.M, tg::kPairBM));
  w.n_seg = static_cast<uint32_t>(ceil_div(p.N, p.epi == tg::kEpiGated ? tg::kGatedTileN : tg::kBN));
  w.n_tiles = w.n_seg * p.segs_n;
  w.k_seg = static_cast<uint32_t>(ceil_div(p.K, tg::kLinBK));
  w.k_blocks = w.k_seg * p.segs_k;
  w.blocks_per_split = (w.k_blocks + splits - 1) / splits;
  w.splits = (w.k_blocks + w.blocks_per_split - 1) / w.blocks_per_split;
  w.units = w.m_tiles * w.n_tiles;
  w.part_rows = static_cast<uint32_t>(ceil_div(p.M, tg::kPartialRows)) * tg::kPartialRows;
  w.part_pitch = static_cast<uint32_t>(ceil_div(p.N, 4)) * 4;   // 16 bytes
  w.partial_bytes = w.splits > 1 || sums ? uint64_t(w.splits) * w.part_rows * w.part_pitch * 4 : 0;
  return w;
}

// What the products' units are expected to take over ``pairs`` CTA pairs, and the joins: the longest
// unit, or every pair's share of all.
double expected_us(const Product* p, const Plan* w, int count, uint32_t pairs) {
  uint32_t at_work = 0;
  for (int i = 0; i < count; ++i) at_work += w[i].units * w[i].splits;
  const double full = at_work < pairs ? double(at_work) / pairs : 1.0;
  const double block = kBlockUs + (kFullBlockUs - kBlockUs) * full;
  double longest = 0, all = 0, join = 0;
  for (int i = 0; i < count; ++i) {
    const double unit = w[i].blocks_per_split * block + kUnitUs;
    const uint32_t units = w[i].units * w[i].splits;
    if (unit > longest) longest = unit;
    all += units * unit;
    if (count == 1) all = ((units + pairs - 1) / pairs) * pairs * unit;   // whole waves
    if (w[i].partial_bytes) {
      const double bytes = double(w[i].splits) * p[i].M * p[i].N * p[i].segs_n * 4.0;
      join = kJoinUs + (join > kJoinUs ? join - kJoinUs : 0) + bytes / kWriteBytes + bytes / kReadBytes;
    }
  }
  return (all / pairs > longest ? all / pairs : longest) + join;
}

// Plans of up to two products in one launch.  Where the units would not fill the pairs, or one product's
// are much longer than a pair's share of all, K may be split at the price of partial sums in fp32 and a
// join: the least expected time decides.  sums: see plan_of, for the first product.
void plan_products(const Product* p, Plan* best, int count, int max_pairs, bool sums = false) {
  const uint32_t pairs = static_cast<uint32_t>(max_pairs);
  uint32_t most[2] = {1, 1};
  for (int i = 0; i < count; ++i) {
    best[i] = plan_of(p[i], 1, i == 0 && sums);
    if (p[i].epi == tg::kEpiStore && best[i].units < pairs) {
      const uint32_t fill = pairs / best[i].units, deep = best[i].k_blocks / kMinBlocks;
      most[i] = fill < deep ? fill : deep;
    }
  }
  double least = expected_us(p, best, count, pairs);
  const uint32_t tries[] = {1, 2, 3, 4, 5, 6, 8, 10, 12, 16, 19, 25, 38, 76};
  for (uint32_t s0 : tries) {
    if (s0 > 1 && s0 > most[0]) break;
    for (uint32_t s1 : tries) {
      if (s1 > 1 && (count < 2 || s1 > most[1])) break;
      if (s0 == 1 && s1 == 1) continue;
      Plan cut[2];
      cut[0] = plan_of(p[0], s0, sums);
      if (count == 2) cut[1] = plan_of(p[1], s1);
      const double us = expected_us(p, cut, count, pairs);
      if (us < least) {
        least = us;
        for (int i = 0; i < count; ++i) best[i] = cut[i];
      }
    }
  }
}

// Few rows: a tile is shared by as many CTAs (a power of two) as it takes for one on every SM, of at least
// two k-blocks of 64 each.  Where 8 do not fill the SMs and have many k-blocks left, K is cut between
// groups first: a CTA has about 0.3 us of a k-block in flight for every one it multiplies, the join of
// the groups' sums takes 3 us.  Measured (bf16, us, one group / groups): gradient towards x of 44 rows,
// 312 columns, 33823 words 33 / 9.
Plan plan_few(const Product& p, int max_pairs) {
  const uint32_t sms = 2 * static_cast<uint32_t>(max_pairs);
  const uint32_t tiles = static_cast<uint32_t>(ceil_div(p.N, tg::kFewM));
  const uint32_t k_blocks = static_cast<uint32_t>(ceil_div(p.K, tg::kFewBK)) * p.segs_k;
  Plan w = plan_of(p, 1);
  w.few = true;
  while (w.ranks < tg::kFewMaxCluster && tiles * w.ranks < sms && k_blocks >= 4 * w.ranks) w.ranks *= 2;
  const uint32_t each = k_blocks / w.ranks;
  if (p.epi == tg::kEpiStore && tiles * w.ranks < sms && each > 20) {
    const uint32_t fill = 2 * sms / (tiles * w.ranks), deep = each / 6;
    w.splits = fill < deep ? fill : deep;
    w.part_rows = static_cast<uint32_t>(p.M);
    if (w.splits > 1) w.partial_bytes = uint64_t(w.splits) * w.part_rows * p.N * 4;
  }
  return w;
}

Plan plan_product(const Product& p, int max_pairs) {
  if (few_rows(p, false)) return plan_few(p, max_pairs);
  Plan w;
  plan_products(&p, &w, 1, max_pairs);
  return w;
}

constexpr uint64_t kWorkspaceAlign = 256;
uint64_t padded(uint64_t bytes) { return ceil_div(bytes, kWorkspaceAlign) * kWorkspaceAlign; }

CUtensorMapDataType type16(int dtype) {
  return dtype == TG_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
}

// The operand ``m`` of a product: boxes of one 64-value atom of K by 128 rows, or of 64 columns by a
// stage's rows of K.
int encode_operand(CUtensorMap* map, const Mat& m, bool mn, int dtype) {
  return encode_tiled(map, type16(dtype), 2, m.p, m.cols, m.rows, 64,
                      mn ? tg::kLinBK : tg::kBM, m.name, true, m.ld * 2);
}

// Enqueues a product with few rows by its plan (without the join of its groups' sums).
int run_few(const Product& p, const Plan& w, char* partials, uint64_t watchdog_ns, int64_t inject,
            cudaStream_t stream) {
  tg::FewLaunch l = {};
  const uint32_t n_pad = tg::few_padded(p.M);
  const int mats = p.epi == tg::kEpiGated || p.segs_k == 2 ? 2 : 1;
  for (int i = 0; i < mats; ++i) {
    const Mat& b = p.b[p.segs_k == 2 ? 2 * i : i];
    TG_TRY(encode_tiled(&l.w[i], type16(p.dtype), 2, b.p, b.cols, b.rows, 64,
                        p.b_mn ? tg::kFewBK : tg::kFewM, b.name, true, b.ld * 2));
    const Mat& x = p.a[p.segs_k == 2 ? i : 0];
    TG_TRY(encode_tiled(&l.x[i], type16(p.dtype), 2, x.p, x.cols, x.rows, 64, n_pad, x.name, true,
                        x.ld * 2));
    if (p.two_terms)
      TG_TRY(encode_tiled(&l.x_rest[i], type16(p.dtype), 2, p.a_rest[i].p, x.cols, x.rows, 64, n_pad,
                          x.name, true, x.ld * 2));
  }
  l.terms = p.two_terms ? 2 : 1;
  l.dtype = p.dtype;
  l.w_mn = p.b_mn;
  l.epi = p.epi;
  l.rows = static_cast<uint32_t>(p.M);
  l.outs = static_cast<uint32_t>(p.N);
  l.tiles = static_cast<uint32_t>(ceil_div(p.N, tg::kFewM));
  l.k_seg = static_cast<uint32_t>(ceil_div(p.K, tg::kFewBK));
  l.k_blocks = l.k_seg * p.segs_k;
  l.ranks = w.ranks;
  l.groups = w.splits;
  l.partials = w.partial_bytes ? reinterpret_cast<float*>(partials) : nullptr;
  l.alpha = p.alpha;
  l.act = p.act;
  l.out = const_cast<void*>(p.c[0].p);
  l.ld_out = p.c[0].ld;
  if (p.epi == tg::kEpiDlogits) l.rest = const_cast<void*>(p.c[1].p);
  if (p.keep) {
    l.g = const_cast<void*>(p.c[1].p);
    l.u = const_cast<void*>(p.c[2].p);
    l.ld_g = p.c[1].ld;
    l.ld_u = p.c[2].ld;
  }
  l.first_col = p.first_col;
  l.slots = p.slots;
  l.stats = p.stats;
  l.hit = p.hit;
  l.lse = p.lse;
  l.loss = p.loss;
  l.watchdog_ns = watchdog_ns ? watchdog_ns : default_watchdog_ns(l.k_blocks);
  l.inject_skip_phase = inject;
  const cudaError_t e = tg::launch_few(l, stream);
  return e == cudaSuccess ? TG_OK : fail_cuda("product launch", e);
}

// What a product's units are to the kernel.  partials: fp32 sums of its N segments, where the plan has
// them.
int encode_product(tg::LinearProduct* l, const Product& p, const Plan& w, char* partials) {
  for (int i = 0; i < p.segs_k; ++i) TG_TRY(encode_operand(&l->a[i], p.a[i], p.a_mn, p.dtype));
  const int across = p.segs_n == 2 || p.epi == tg::kEpiGated ? 2 : 1;
  for (int k = 0; k < p.segs_k; ++k)
    for (int i = 0; i < across; ++i)
      TG_TRY(encode_operand(&l->b[2 * k + i], p.b[2 * k + i], p.b_mn, p.dtype));
  l->partial = 0;
  if (w.partial_bytes) {
    for (int i = 0; i < p.segs_n; ++i)
      TG_TRY(encode_tiled(&l->c[i], CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 4,
                          partials + i * padded(w.partial_bytes), p.N,
                          uint64_t(w.splits) * w.part_rows, 32, tg::kPartialRows, "workspace", true,
                          uint64_t(w.part_pitch) * 4));
    l->partial = p.accumulate == 2 ? 2 : 1;
  } else {
    for (int i = 0; i < 3; ++i)
      if (p.c[i].p)
        TG_TRY(encode_tiled(&l->c[i], type16(p.dtype), 2, p.c[i].p, p.c[i].cols, p.c[i].rows,
                            tg::kEpiN, 32, p.c[i].name, true, p.c[i].ld * 2));
  }
  l->a_mn = p.a_mn;
  l->b_mn = p.b_mn;
  l->M = static_cast<uint32_t>(p.M);
  l->N = static_cast<uint32_t>(p.N);
  l->m_blocks = w.m_tiles;
  l->n_blocks = w.n_tiles;
  l->k_blocks = w.k_blocks;
  l->n_seg = w.n_seg;
  l->k_seg = w.k_seg;
  // All of an operand that fits in a quarter of the L2 stays there: tiles go along it, so that the other
  // one is read once.  Measured (bf16, us, along it / in groups of 8): gradients of 4096 x 4096 x 65536
  // (33 MB) 3575 / 3627, but the gated projections 8192 x 4096 x 8192 with g and u (67 MB) 617 / 579.
  const uint64_t k2 = uint64_t(p.K) * p.segs_k * 2, fits = 32u << 20;
  if (k2 * p.N * (p.epi == tg::kEpiGated ? 2 : p.segs_n) <= fits) {
    l->group = w.n_tiles;
    l->column_major = 0;
  } else if (k2 * p.M <= fits) {
    l->group = w.m_tiles;
    l->column_major = 1;
  } else {
    l->group = tg::kGroup;
    l->column_major = 0;
  }
  l->split_from = l->total_units = w.units;
  l->splits = w.splits;
  l->blocks_per_split = w.blocks_per_split;
  l->part_rows = w.part_rows;
  l->segment_log = p.logits ? tg::kLogitSegmentLog : tg::kLinSegmentLog;
  l->alpha = p.alpha;
  return TG_OK;
}

// Enqueues up to two products in one launch, the one with the longer units first.
int run_products(const Product* p, const Plan* w, char* const* partials, int count, int max_pairs,
                 uint64_t watchdog_ns, int64_t inject, cudaStream_t stream) {
  tg::LinearLaunch l = {};
  const uint32_t pairs = static_cast<uint32_t>(max_pairs);
  const int first = count == 2 && w[1].blocks_per_split > w[0].blocks_per_split ? 1 : 0;
  uint32_t units = 0, k_blocks = 0;
  for (int i = 0; i < count; ++i) {
    const int at = first ? 1 - i : i;
    TG_TRY(encode_product(&l.q[i], p[at], w[at], partials[at]));
    units += w[at].units * w[at].splits;
    k_blocks = w[at].k_blocks > k_blocks ? w[at].k_blocks : k_blocks;
  }
  // Workers without a unit in the first product's last round take units of the second one meanwhile
  // (LinearUnits), and the rounds go through what is left.  Where their last one would keep at most
  // half of the pairs busy, its tiles are cut in halves.
  tg::LinearProduct& last = l.q[count - 1];
  uint32_t workers = units < pairs ? units : pairs, ahead = 0;
  if (count == 2) {
    const uint32_t idle = workers - l.q[0].total_units * l.q[0].splits % workers;
    if (idle < workers) {
      const uint32_t as_long = l.q[0].blocks_per_split / last.blocks_per_split;
      const uint32_t share = (last.total_units * last.splits + idle - 1) / idle;
      l.extra = as_long < share ? as_long : share;
      ahead = idle * l.extra;
    }
  }
  if (last.splits == 1 && last.total_units > ahead && (count == 1 || units >= pairs)) {
    uint32_t from, all;
    tg::PersistentTileScheduler::tail_split(last.total_units - ahead, pairs, from, all);
    last.split_from = ahead + from;
    last.total_units = ahead + all;
    if (count == 1) workers = all < pairs ? all : pairs;
  }
  l.products = count;
  l.dtype = p[0].dtype;
  l.epi = p[0].epi;
  l.act = p[0].act;
  l.keep = p[0].keep;
  l.first_col = p[0].first_col;
  l.slots = p[0].slots;
  l.stats = p[0].stats;
  l.hit = p[0].hit;
  l.lse = p[0].lse;
  l.loss = p[0].loss;
  l.grid = 2 * workers;
  // a k-block of this kernel is two of the 64-deep ones that the default limit counts
  l.watchdog_ns = watchdog_ns ? watchdog_ns : default_watchdog_ns(2 * k_blocks);
  l.inject_skip_phase = inject;
  const cudaError_t e = tg::launch_linear(l, stream);
  return e == cudaSuccess ? TG_OK : fail_cuda("product launch", e);
}

// Adds the partial sums of the products that have them into their outputs, in one launch.
int join_products(const Product* p, const Plan* w, char* const* partials, int count, int sms,
                  cudaStream_t stream) {
  tg::LinearJoin jobs[3];
  int n = 0;
  for (int q = 0; q < count; ++q)
    for (int i = 0; i < p[q].segs_n && w[q].partial_bytes; ++i) {
      tg::LinearJoin& j = jobs[n++];
      j.partials = reinterpret_cast<const float*>(partials[q] + i * padded(w[q].partial_bytes));
      j.splits = w[q].splits;
      j.part_rows = w[q].part_rows;
      j.rows = static_cast<uint32_t>(p[q].M);
      j.cols = static_cast<uint32_t>(p[q].N);
      j.alpha = p[q].alpha;
      j.out = const_cast<void*>(p[q].c[i].p);
      j.ld_out = p[q].c[i].ld;
    }
  if (n == 0) return TG_OK;
  const cudaError_t e = tg::launch_linear_join(jobs, n, p[0].dtype, sms, stream);
  return e == cudaSuccess ? TG_OK : fail_cuda("join launch", e);
}

uint64_t partials_of(const Product& p, const Plan& w) {
  return w.partial_bytes ? p.segs_n * padded(w.partial_bytes) : 0;
}

// A product by itself: its units, and the join of its partial sums at ``ws`` where it has them.
int whole_product(const Product& p, const Plan& w, void* ws, int sms, int pairs, cudaStream_t stream,
                  uint64_t watchdog_ns = 0, int64_t inject = -1) {
  char* const partials[1] = {static_cast<char*>(ws)};
  if (w.few)
    TG_TRY(run_few(p, w, partials[0], watchdog_ns, inject, stream));
  else
    TG_TRY(run_products(&p, &w, partials, 1, pairs, watchdog_ns, inject, stream));
  return join_products(&p, &w, partials, 1, sms, stream);
}

// The gradients towards an input and towards weights that are taken from the same matrices: p[0] and
// p[1] in one launch, or p[0] by the kernel for few rows.  sums: p[0]'s fp32 sums run over several
// launches and are joined by the caller.
struct GradPlans {
  Plan w[2];
  uint64_t bytes[2];        // partial sums of each

  GradPlans(const Product* p, int pairs, bool sums = false) {
    if (few_rows(p[0], sums)) {
      w[0] = plan_product(p[0], pairs);
      if (p[1].K <= tg::kTwoTermRows) {
        w[1] = plan_of(p[1], 1);
        w[1].outer = true;
      } else {
        plan_products(&p[1], &w[1], 1, pairs);
      }
    } else {
      plan_products(p, w, 2, pairs, sums);
    }
    for (int i = 0; i < 2; ++i) bytes[i] = partials_of(p[i], w[i]);
  }
};

// Enqueues a gradient towards weights from at most 8 rows: p.K of them, a_mn and b_mn.
int run_outer(const Product& p, int sms, cudaStream_t stream) {
  tg::OuterLaunch l = {};
  l.a = p.a[0].p;
  l.a_rest = p.a_rest[0].p;
  l.ld_a = p.a[0].ld;
  l.ld_b = p.b[0].ld;
  l.results = p.segs_n;
  for (int i = 0; i < p.segs_n; ++i) {
    l.b[i] = p.b[i].p;
    l.b_rest[i] = p.b_rest[i].p;
    l.out[i] = const_cast<void*>(p.c[i].p);
    l.ld_out[i] = p.c[i].ld;
  }
  l.rows = static_cast<uint32_t>(p.K);
  l.m = static_cast<uint32_t>(p.M);
  l.n = static_cast<uint32_t>(p.N);
  l.alpha = p.alpha;
  l.dtype = p.dtype;
  l.sms = sms;
  const cudaError_t e = tg::launch_outer(l, stream);
  return e == cudaSuccess ? TG_OK : fail_cuda("product launch", e);
}

// Enqueues what is asked for of the two.  Their plans hold for both together and for either.
int run_grads(const Product* p, const GradPlans& o, const bool (&wanted)[2], bool join_first,
              char* const* partials, int sms, int pairs, cudaStream_t stream) {
  Product q[2];
  Plan w[2];
  char* at[2];
  int n = 0;
  for (int i = 0; i < 2; ++i) {
    if (!wanted[i]) continue;
    q[n] = p[i];
    w[n] = o.w[i];
    at[n++] = partials[i];
  }
  if (n == 0) return TG_OK;
  const int few = w[0].few ? 1 : 0;   // the second one never is
  if (few) TG_TRY(run_few(q[0], w[0], at[0], 0, -1, stream));
  if (n > few && w[n - 1].outer)
    TG_TRY(run_outer(q[n - 1], sms, stream));
  else if (n > few)
    TG_TRY(run_products(q + few, w + few, at + few, n - few, pairs, 0, -1, stream));
  const int skip = wanted[0] && !join_first ? 1 : 0;
  return join_products(q + skip, w + skip, at + skip, n - skip, sms, stream);
}

// ---------------------------------------------------------------- checks
int check_dtype16(int dtype) {
  if (dtype != TG_F16 && dtype != TG_BF16) return fail(TG_ERR_ARG, "unknown dtype %d", dtype);
  return TG_OK;
}

// Sizes of a layer: multiples of 8 along the contiguous rows of every matrix.
int check_layer(int64_t rows, int64_t cols, int64_t outs) {
  TG_TRY(check_sizes(rows, cols));
  if (outs < 0 || outs > kMaxDim)
    return fail(TG_ERR_ARG, "outs=%lld must be in [0, 2^31)", (long long)outs);
  if (cols % 8 != 0 || outs % 8 != 0)
    return fail(TG_ERR_ALIGN, "cols=%lld and outs=%lld must be multiples of 8 (16-byte rows)",
                (long long)cols, (long long)outs);
  return TG_OK;
}

int check_tiles(int64_t m, int64_t n, int64_t segs = 1) {
  if (ceil_div(m, 128) * ceil_div(n, 128) * segs > static_cast<uint64_t>(kMaxDim))
    return fail(TG_ERR_ARG, "too many output tiles");
  return TG_OK;
}

struct Ld {
  int64_t ld, cols;
  const char* name;
};
int check_lds(std::initializer_list<Ld> lds) {
  for (const Ld& l : lds) {
    TG_TRY(check_ld(l.ld, l.cols, l.name));
    if (l.ld % 8 != 0)
      return fail(TG_ERR_ALIGN, "%s=%lld must be a multiple of 8 (16-byte rows)", l.name,
                  (long long)l.ld);
  }
  return TG_OK;
}

int check_mats(std::initializer_list<Mat> mats) {
  for (const Mat& m : mats)
    if (m.rows > 0 && m.cols > 0) TG_TRY(check_array(m.p, 16, m.name));
  return TG_OK;
}

Region region(const Mat& m) {
  return matrix(m.rows > 0 && m.cols > 0 ? m.p : nullptr, m.rows, m.cols, m.ld, 2, m.name);
}

int check_workspace(const void* ws, int64_t bytes, uint64_t need) {
  if (bytes < 0) return fail(TG_ERR_ARG, "negative workspace size");
  if (need == 0) return TG_OK;
  if (!ws || static_cast<uint64_t>(bytes) < need)
    return fail(TG_ERR_ARG, "workspace of %lld bytes; this call needs %llu",
                (long long)(ws ? bytes : 0), (unsigned long long)need);
  return check_array(ws, kWorkspaceAlign, "workspace");
}

// C = 0 for a matrix with 16-bit values
int zero_fill(const Mat& m, cudaStream_t stream) {
  if (m.rows == 0 || m.cols == 0) return TG_OK;
  const cudaError_t e =
      cudaMemset2DAsync(const_cast<void*>(m.p), m.ld * 2, 0, m.cols * 2, m.rows, stream);
  return e == cudaSuccess ? TG_OK : fail_cuda("zero fill", e);
}

int watchdog_result(cudaStream_t stream) {
  unsigned int word = 0;
  const cudaError_t e = tg::read_and_clear_watchdog_status(&word, stream);
  if (e != cudaSuccess) return fail_cuda("execution", e);
  if (word)
    return fail(TG_ERR_TIMEOUT, "watchdog: a wait gave up (roles 0x%x: 1 producer, 2 MMA, "
                "4 epilogue, 8 shutdown)", word);
  return TG_OK;
}

// ---------------------------------------------------------------- input gradient
// dX [rows, cols] = dY [rows, outs] W^T, W [cols, outs]: K = outs, contiguous in both operands
Product input_grad_product(const Mat& dy, const Mat& w, const Mat& dx, int dtype) {
  Product p;
  p.dtype = dtype;
  p.M = dx.rows;
  p.N = dx.cols;
  p.K = dy.cols;
  p.a[0] = dy;
  p.b[0] = w;
  p.c[0] = dx;
  return p;
}

int input_grad_impl(const void* dy, const void* w, void* dx, int64_t rows, int64_t cols,
                    int64_t outs, int64_t ld_dy, int64_t ld_w, int64_t ld_dx, int dtype, void* ws,
                    int64_t ws_bytes, void* stream, bool debug, uint64_t watchdog_ns,
                    int64_t inject) {
  TG_TRY(check_dtype16(dtype));
  TG_TRY(check_layer(rows, cols, outs));
  TG_TRY(check_tiles(rows, cols));
  TG_TRY(check_lds({{ld_dy, outs, "ld_dy"}, {ld_w, outs, "ld_w"}, {ld_dx, cols, "ld_dx"}}));
  TG_TRY(check_workspace(nullptr, ws_bytes, 0));
  if (rows == 0 || cols == 0) return TG_OK;
  const Mat mdy = {dy, rows, outs, ld_dy, "dY"}, mw = {w, cols, outs, ld_w, "W"},
            mdx = {dx, rows, cols, ld_dx, "dX"};
  TG_TRY(check_mats({mdx, mdy, mw}));
  int sms = 0, pairs = 0;
  TG_TRY(linear_ready(&sms, &pairs));
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (outs == 0) return zero_fill(mdx, st);
  const Product p = input_grad_product(mdy, mw, mdx, dtype);
  const Plan plan = plan_product(p, pairs);
  const uint64_t need = partials_of(p, plan);
  TG_TRY(check_workspace(ws, ws_bytes, need));
  const Region r[] = {region(mdx), {need ? ws : nullptr, need, "workspace"}, region(mdy), region(mw)};
  TG_TRY(check_apart(r, 2, 4));
  if (debug) {
    const cudaError_t e = tg::clear_watchdog_status(st);
    if (e != cudaSuccess) return fail_cuda("clearing the watchdog word", e);
  }
  TG_TRY(whole_product(p, plan, ws, sms, pairs, st, watchdog_ns, inject));
  return debug ? watchdog_result(st) : TG_OK;
}

// ---------------------------------------------------------------- gated feed-forward projections
int check_act(int act) {
  if (act != TG_ACT_SILU && act != TG_ACT_GELU)
    return fail(TG_ERR_ARG, "unknown activation %d", act);
  return TG_OK;
}

// g and u by one MMA side by side, or, with K split, as two N segments whose sums are joined
struct GatedPlan {
  Product p;
  Plan plan;
};
GatedPlan gated_plan(const Mat& x, const Mat& wg, const Mat& wu, const Mat& h, int dtype,
                     int pairs) {
  GatedPlan o;
  Product& p = o.p;
  p.epi = tg::kEpiGated;
  p.dtype = dtype;
  p.b_mn = true;
  p.M = x.rows;
  p.N = h.cols;
  p.K = x.cols;
  p.a[0] = x;
  p.b[0] = wg;
  p.b[1] = wu;
  p.c[0] = h;
  o.plan = plan_product(p, pairs);
  if (o.plan.few) return o;
  Product two = p;
  two.epi = tg::kEpiStore;
  two.segs_n = 2;
  Plan cut;
  plan_products(&two, &cut, 1, pairs);
  if (cut.splits > 1 && expected_us(&two, &cut, 1, pairs) < expected_us(&p, &o.plan, 1, pairs)) {
    o.p = two;
    o.plan = cut;
  }
  return o;
}

// Gradients that are rounded to 16 bits on the way to both products: with few rows their errors do not
// average out, so they come in two terms (tg_few_kernel.cuh, tg_outer_kernel.cuh).
bool two_terms(int64_t rows) { return rows <= tg::kTwoTermRows; }

struct GatedBwd {
  Product p[2];             // dx; dwg and dwu
  GradPlans plans;
  uint64_t dgu_bytes, total;   // dgu_bytes: of one term
};
// In front of dg and du: the largest values of their blocks, and the factor that undoes their scale (fp16)
constexpr uint64_t kGradTopsBytes = tg::kGradBlocks * 4, kGradScaleBytes = kGradTopsBytes + kWorkspaceAlign;
// With null pointers where only sizes matter.
GatedBwd gated_bwd_plan(const Mat& x, const Mat& wg, const Mat& wu, const Mat& dx, const Mat& dwg,
                        const Mat& dwu, void* dgu, int dtype, int pairs) {
  const int64_t rows = x.rows, cols = x.cols, outs = wg.cols;
  const uint64_t dgu_bytes = padded(uint64_t(rows) * 2 * outs * 2);
  const bool two = two_terms(rows);
  // dg or du of a term
  auto part = [&](int term, int which) {
    char* at = dgu ? static_cast<char*>(dgu) + term * dgu_bytes + which * 2 * outs : nullptr;
    return Mat{at, rows, outs, 2 * outs, which ? "du" : "dg"};
  };
  Product p[2];
  // dX = dg Wg^T + du Wu^T: K in two segments
  p[0].dtype = dtype;
  p[0].M = rows;
  p[0].N = cols;
  p[0].K = outs;
  p[0].segs_k = 2;
  p[0].b[0] = wg;
  p[0].b[2] = wu;
  p[0].c[0] = dx;
  p[0].two_terms = two;
  // dWg = X^T dg, dWu = X^T du: N in two segments
  p[1].dtype = dtype;
  p[1].a_mn = p[1].b_mn = true;
  p[1].M = cols;
  p[1].N = outs;
  p[1].K = rows;
  p[1].segs_n = 2;
  p[1].a[0] = x;
  p[1].c[0] = dwg;
  p[1].c[1] = dwu;
  for (int i = 0; i < 2; ++i) {
    p[0].a[i] = p[1].b[i] = part(0, i);
    if (two) p[0].a_rest[i] = p[1].b_rest[i] = part(1, i);
  }
  GatedBwd o = {{p[0], p[1]}, GradPlans(p, pairs), dgu_bytes, 0};
  o.total = kGradScaleBytes + (two ? 2 : 1) * dgu_bytes + o.plans.bytes[0] + o.plans.bytes[1];
  return o;
}

// ---------------------------------------------------------------- cross entropy
constexpr uint64_t kXentChunkBytes = 256u << 20;   // gradients of logits held at a time
constexpr int64_t kXentMinChunk = 2048;

int check_xent(int64_t rows, int64_t cols, int64_t vocab, int64_t ld_x, int64_t ld_w, int dtype) {
  TG_TRY(check_dtype16(dtype));
  TG_TRY(check_sizes(rows, cols));
  if (vocab < 1 || vocab > kMaxDim)
    return fail(TG_ERR_ARG, "vocab=%lld must be in [1, 2^31)", (long long)vocab);
  if (cols == 0) return fail(TG_ERR_ARG, "cols must be at least 8");
  if (cols % 8 != 0)
    return fail(TG_ERR_ALIGN, "cols=%lld must be a multiple of 8 (16-byte rows)", (long long)cols);
  TG_TRY(check_lds({{ld_x, cols, "ld_x"}, {ld_w, cols, "ld_w"}}));
  return check_tiles(rows, vocab);
}

// logits of columns [first, first + n) of the vocabulary, W's rows
Product logits_product(int epi, const Mat& x, const Mat& w, int64_t first, int64_t n,
                       const tg::XentRows& loss, int dtype) {
  Product p;
  p.epi = epi;
  p.logits = true;
  p.dtype = dtype;
  p.M = x.rows;
  p.N = n;
  p.K = x.cols;
  p.a[0] = x;
  p.b[0] = {static_cast<const char*>(w.p) + first * w.ld * 2, n, w.cols, w.ld, w.name};
  p.loss = loss;
  p.first_col = static_cast<uint32_t>(first);
  return p;
}

// How logits are made: by an epilogue of the product, or, where few tiles have long sums, from the parts
// of split sums.
struct LogitsPlan {
  Product p;                // with kEpiStore: parts
  Plan plan;
  uint64_t part_bytes;
};
LogitsPlan logits_plan(const Product& p, int pairs) {
  LogitsPlan o = {p, plan_product(p, pairs), 0};
  if (o.plan.few) return o;
  Product parts = p;
  parts.epi = tg::kEpiStore;
  Plan cut;
  plan_products(&parts, &cut, 1, pairs);
  if (cut.splits > 1 && expected_us(&parts, &cut, 1, pairs) < expected_us(&p, &o.plan, 1, pairs)) {
    o.p = parts;
    o.plan = cut;
    o.part_bytes = partials_of(parts, cut);
  }
  return o;
}
tg::XentParts parts_of(const Plan& w, const char* parts) {
  return {reinterpret_cast<const float*>(parts), w.splits, w.part_rows, w.part_pitch};
}

struct XentFwd {
  LogitsPlan logits;
  uint32_t slots;
  uint64_t stats_bytes, total;
};
XentFwd xent_fwd_plan(const Mat& x, const Mat& w, const tg::XentRows& loss, int dtype, int pairs) {
  XentFwd o;
  o.logits = logits_plan(logits_product(tg::kEpiStats, x, w, 0, w.rows, loss, dtype), pairs);
  o.slots = static_cast<uint32_t>(ceil_div(w.rows, o.logits.plan.few ? tg::kFewM : tg::kStatCols));
  o.stats_bytes = padded(uint64_t(x.rows) * o.slots * 8);
  o.total = o.logits.part_bytes ? o.logits.part_bytes
                                : o.stats_bytes + padded(uint64_t(x.rows) * 4);
  return o;
}

// The gradients, a piece of ``chunk`` columns of the vocabulary at a time: the gradients of the piece's
// logits, its rows of dW, and its share of dX, whose fp32 sums run over the pieces.
struct XentBwd {
  int64_t chunk, chunks;
  bool sums;                // dX is summed in fp32 over the pieces
  bool two;                 // the gradients of the logits come in two terms
  uint64_t dl_bytes;        // of one term
  uint64_t part_bytes, dx_bytes, dw_bytes, total;
};

// rest: the second term of dl, or null
Product xent_dx_product(const Mat& dl, const Mat* rest, const Mat& w, int64_t first, const Mat& dx,
                        int dtype) {
  Product p;
  p.two_terms = rest != nullptr;
  if (rest) p.a_rest[0] = *rest;
  p.dtype = dtype;
  p.b_mn = true;
  p.M = dl.rows;
  p.N = dx.cols;
  p.K = dl.cols;
  p.a[0] = dl;
  p.b[0] = {static_cast<const char*>(w.p) + first * w.ld * 2, dl.cols, w.cols, w.ld, w.name};
  p.c[0] = dx;
  return p;
}

Product xent_dw_product(const Mat& dl, const Mat* rest, const Mat& x, const Mat& dw, int64_t first,
                        int dtype) {
  Product p;
  if (rest) p.a_rest[0] = *rest;
  p.dtype = dtype;
  p.a_mn = p.b_mn = true;
  p.M = dl.cols;
  p.N = x.cols;
  p.K = dl.rows;
  p.a[0] = dl;
  p.b[0] = x;
  p.c[0] = {static_cast<const char*>(dw.p) + first * dw.ld * 2, dl.cols, dw.cols, dw.ld, dw.name};
  return p;
}

XentBwd xent_bwd_plan(int64_t rows, int64_t cols, int64_t vocab, int dtype, int pairs) {
  XentBwd o;
  int64_t most = static_cast<int64_t>(kXentChunkBytes / (uint64_t(rows) * 2)) / tg::kBN * tg::kBN;
  if (most < kXentMinChunk) most = kXentMinChunk;
  o.chunks = static_cast<int64_t>(ceil_div(vocab, most));
  o.chunk = static_cast<int64_t>(ceil_div(ceil_div(vocab, o.chunks), tg::kBN)) * tg::kBN;
  o.chunks = static_cast<int64_t>(ceil_div(vocab, o.chunk));
  o.sums = o.chunks > 1;
  o.two = two_terms(rows) && !o.sums;
  o.dl_bytes = padded(uint64_t(rows) * o.chunk * 2);
  o.part_bytes = o.dx_bytes = o.dw_bytes = 0;
  const Mat x = {nullptr, rows, cols, cols, ""}, w = {nullptr, vocab, cols, cols, ""};
  // the last piece may be narrower and split its tokens more finely
  for (const int64_t first : {int64_t(0), (o.chunks - 1) * o.chunk}) {
    const Mat dl = {nullptr, rows, vocab - first < o.chunk ? vocab - first : o.chunk, o.chunk, ""};
    const Mat* rest = o.two ? &dl : nullptr;
    const Product p[2] = {xent_dx_product(dl, rest, w, first, x, dtype),
                          xent_dw_product(dl, rest, x, w, first, dtype)};
    const GradPlans plans(p, pairs, o.sums);
    const LogitsPlan logits =
        logits_plan(logits_product(tg::kEpiDlogits, x, w, first, dl.cols, {}, dtype), pairs);
    if (logits.part_bytes > o.part_bytes) o.part_bytes = logits.part_bytes;
    if (first == 0) o.dx_bytes = plans.bytes[0];
    if (plans.bytes[1] > o.dw_bytes) o.dw_bytes = plans.bytes[1];
  }
  o.total = (o.two ? 2 : 1) * o.dl_bytes + kWorkspaceAlign + o.part_bytes + o.dx_bytes +
            o.dw_bytes;
  return o;
}

}  // namespace

extern "C" {

int64_t tg_input_grad_workspace_bytes(int64_t rows, int64_t cols, int64_t outs) {
  TG_TRY(check_layer(rows, cols, outs));
  TG_TRY(check_tiles(rows, cols));
  if (rows == 0 || cols == 0 || outs == 0) return 0;
  int pairs = 0;
  TG_TRY(linear_ready(nullptr, &pairs));
  const Product p = input_grad_product({nullptr, rows, outs, outs, ""}, {nullptr, cols, outs, outs, ""},
                                       {nullptr, rows, cols, cols, ""}, TG_BF16);
  return static_cast<int64_t>(partials_of(p, plan_product(p, pairs)));
}

int tg_input_grad(const void* dY_dev, const void* W_dev, void* dX_dev, int64_t rows, int64_t cols,
                  int64_t outs, int64_t ld_dy, int64_t ld_w, int64_t ld_dx, int dtype,
                  void* workspace_dev, int64_t workspace_bytes, void* stream) {
  return input_grad_impl(dY_dev, W_dev, dX_dev, rows, cols, outs, ld_dy, ld_w, ld_dx, dtype,
                         workspace_dev, workspace_bytes, stream, false, 0, -1);
}

int tg_input_grad_debug(const void* dY_dev, const void* W_dev, void* dX_dev, int64_t rows,
                        int64_t cols, int64_t outs, int64_t ld_dy, int64_t ld_w, int64_t ld_dx,
                        int dtype, void* workspace_dev, int64_t workspace_bytes, void* stream,
                        uint64_t watchdog_ns, int64_t inject_skip_phase) {
  return input_grad_impl(dY_dev, W_dev, dX_dev, rows, cols, outs, ld_dy, ld_w, ld_dx, dtype,
                         workspace_dev, workspace_bytes, stream, true, watchdog_ns,
                         inject_skip_phase);
}

int64_t tg_gated_fwd_workspace_bytes(int64_t rows, int64_t cols, int64_t outs) {
  TG_TRY(check_layer(rows, cols, outs));
  TG_TRY(check_tiles(rows, outs, 2));
  if (rows == 0 || cols == 0 || outs == 0) return 0;
  int pairs = 0;
  TG_TRY(linear_ready(nullptr, &pairs));
  const Mat w = {nullptr, cols, outs, outs, ""};
  const GatedPlan o = gated_plan({nullptr, rows, cols, cols, ""}, w, w,
                                 {nullptr, rows, outs, outs, ""}, TG_BF16, pairs);
  return static_cast<int64_t>(partials_of(o.p, o.plan));
}

int tg_gated_fwd(const void* x_dev, const void* wg_dev, const void* wu_dev, void* h_dev,
                 void* g_dev, void* u_dev, int64_t rows, int64_t cols, int64_t outs, int64_t ld_x,
                 int64_t ld_wg, int64_t ld_wu, int64_t ld_h, int64_t ld_g, int64_t ld_u, int act,
                 int dtype, void* workspace_dev, int64_t workspace_bytes, void* stream) {
  TG_TRY(check_dtype16(dtype));
  TG_TRY(check_act(act));
  TG_TRY(check_layer(rows, cols, outs));
  TG_TRY(check_tiles(rows, outs, 2));
  const bool keep = g_dev || u_dev;
  if (keep && !(g_dev && u_dev)) return fail(TG_ERR_ARG, "g and u are kept together or not at all");
  TG_TRY(check_lds({{ld_x, cols, "ld_x"}, {ld_wg, outs, "ld_wg"}, {ld_wu, outs, "ld_wu"},
                    {ld_h, outs, "ld_h"}}));
  if (keep) TG_TRY(check_lds({{ld_g, outs, "ld_g"}, {ld_u, outs, "ld_u"}}));
  TG_TRY(check_workspace(nullptr, workspace_bytes, 0));
  if (rows == 0 || outs == 0) return TG_OK;
  const Mat x = {x_dev, rows, cols, ld_x, "x"}, wg = {wg_dev, cols, outs, ld_wg, "wg"},
            wu = {wu_dev, cols, outs, ld_wu, "wu"}, h = {h_dev, rows, outs, ld_h, "h"},
            g = {g_dev, keep ? rows : 0, outs, ld_g, "g"}, u = {u_dev, keep ? rows : 0, outs, ld_u, "u"};
  TG_TRY(check_mats({h, g, u, x, wg, wu}));
  int sms = 0, pairs = 0;
  TG_TRY(linear_ready(&sms, &pairs));
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (cols == 0) {
    for (const Mat& m : {h, g, u}) TG_TRY(zero_fill(m, st));
    return TG_OK;
  }
  GatedPlan o = gated_plan(x, wg, wu, h, dtype, pairs);
  const uint64_t need = partials_of(o.p, o.plan);
  TG_TRY(check_workspace(workspace_dev, workspace_bytes, need));
  const Region r[] = {region(h), region(g), region(u), {need ? workspace_dev : nullptr, need, "workspace"},
                      region(x), region(wg), region(wu)};
  TG_TRY(check_apart(r, 4, 7));
  if (!need) {
    o.p.act = act;
    o.p.keep = keep;
    o.p.c[1] = g;
    o.p.c[2] = u;
    return whole_product(o.p, o.plan, nullptr, sms, pairs, st);
  }
  char* const partials[1] = {static_cast<char*>(workspace_dev)};
  TG_TRY(run_products(&o.p, &o.plan, partials, 1, pairs, 0, -1, st));
  tg::GatedJoin j;
  j.g_parts = reinterpret_cast<const float*>(partials[0]);
  j.u_parts = reinterpret_cast<const float*>(partials[0] + padded(o.plan.partial_bytes));
  j.splits = o.plan.splits;
  j.part_rows = o.plan.part_rows;
  j.rows = static_cast<uint32_t>(rows);
  j.outs = static_cast<uint32_t>(outs);
  j.act = act;
  j.h = h_dev;
  j.g = g_dev;
  j.u = u_dev;
  j.ld_h = ld_h;
  j.ld_g = ld_g;
  j.ld_u = ld_u;
  j.dtype = dtype;
  j.sms = sms;
  const cudaError_t e = tg::launch_gated_join(j, st);
  return e == cudaSuccess ? TG_OK : fail_cuda("join launch", e);
}

int64_t tg_gated_bwd_workspace_bytes(int64_t rows, int64_t cols, int64_t outs) {
  TG_TRY(check_layer(rows, cols, outs));
  TG_TRY(check_tiles(rows, cols));
  TG_TRY(check_tiles(cols, outs, 2));
  if (rows == 0 || cols == 0 || outs == 0) return 0;
  int pairs = 0;
  TG_TRY(linear_ready(nullptr, &pairs));
  const Mat x = {nullptr, rows, cols, cols, ""}, w = {nullptr, cols, outs, outs, ""};
  return static_cast<int64_t>(gated_bwd_plan(x, w, w, x, w, w, nullptr, TG_BF16, pairs).total);
}

int tg_gated_bwd(const void* dh_dev, const void* g_dev, const void* u_dev, const void* x_dev,
                 const void* wg_dev, const void* wu_dev, void* dx_dev, void* dwg_dev, void* dwu_dev,
                 int64_t rows, int64_t cols, int64_t outs, int64_t ld_dh, int64_t ld_g,
                 int64_t ld_u, int64_t ld_x, int64_t ld_wg, int64_t ld_wu, int64_t ld_dx,
                 int64_t ld_dwg, int64_t ld_dwu, int act, int dtype, void* workspace_dev,
                 int64_t workspace_bytes, void* stream) {
  TG_TRY(check_dtype16(dtype));
  TG_TRY(check_act(act));
  TG_TRY(check_layer(rows, cols, outs));
  TG_TRY(check_tiles(rows, cols));
  TG_TRY(check_tiles(cols, outs, 2));
  const bool weights = dwg_dev || dwu_dev;
  if (weights && !(dwg_dev && dwu_dev))
    return fail(TG_ERR_ARG, "dwg and dwu are asked for together or not at all");
  TG_TRY(check_lds({{ld_dh, outs, "ld_dh"}, {ld_g, outs, "ld_g"}, {ld_u, outs, "ld_u"}}));
  if (weights)
    TG_TRY(check_lds({{ld_x, cols, "ld_x"}, {ld_dwg, outs, "ld_dwg"}, {ld_dwu, outs, "ld_dwu"}}));
  if (dx_dev)
    TG_TRY(check_lds({{ld_wg, outs, "ld_wg"}, {ld_wu, outs, "ld_wu"}, {ld_dx, cols, "ld_dx"}}));
  TG_TRY(check_workspace(nullptr, workspace_bytes, 0));
  if (cols == 0 || (!dx_dev && !weights)) return TG_OK;
  const int64_t x_rows = weights ? rows : 0, w_rows = dx_dev ? cols : 0;
  const Mat dh = {dh_dev, rows, outs, ld_dh, "dh"}, g = {g_dev, rows, outs, ld_g, "g"},
            u = {u_dev, rows, outs, ld_u, "u"}, x = {x_dev, x_rows, cols, ld_x, "x"},
            wg = {wg_dev, w_rows, outs, ld_wg, "wg"}, wu = {wu_dev, w_rows, outs, ld_wu, "wu"},
            dx = {dx_dev, dx_dev ? rows : 0, cols, ld_dx, "dx"},
            dwg = {dwg_dev, weights ? cols : 0, outs, ld_dwg, "dwg"},
            dwu = {dwu_dev, weights ? cols : 0, outs, ld_dwu, "dwu"};
  TG_TRY(check_mats({dx, dwg, dwu, dh, g, u, x, wg, wu}));
  int sms = 0, pairs = 0;
  TG_TRY(linear_ready(&sms, &pairs));
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (rows == 0 || outs == 0) {
    for (const Mat& m : {dx, dwg, dwu}) TG_TRY(zero_fill(m, st));
    return TG_OK;
  }
  const Mat sx = {x_dev, rows, cols, ld_x, "x"}, swg = {wg_dev, cols, outs, ld_wg, "wg"},
            swu = {wu_dev, cols, outs, ld_wu, "wu"};   // sizes whether asked for or not
  char* const scale = static_cast<char*>(workspace_dev);
  char* const dgu = scale ? scale + kGradScaleBytes : nullptr;
  GatedBwd o = gated_bwd_plan(sx, swg, swu, dx, dwg, dwu, dgu, dtype, pairs);
  TG_TRY(check_workspace(workspace_dev, workspace_bytes, o.total));
  const Region r[] = {region(dx), region(dwg), region(dwu), {workspace_dev, o.total, "workspace"},
                      region(dh), region(g), region(u), region(x), region(wg), region(wu)};
  TG_TRY(check_apart(r, 4, 10));
  tg::GatedGrad e;
  e.dh = dh_dev;
  e.g = g_dev;
  e.u = u_dev;
  e.dgu = dgu;
  e.rest = two_terms(rows) ? dgu + o.dgu_bytes : nullptr;
  e.tops = reinterpret_cast<float*>(scale);
  e.alpha = reinterpret_cast<float*>(scale + kGradTopsBytes);
  if (dtype == TG_F16) o.p[0].alpha = o.p[1].alpha = e.alpha;
  e.rows = rows;
  e.outs = outs;
  e.ld_dh = ld_dh;
  e.ld_g = ld_g;
  e.ld_u = ld_u;
  e.act = act;
  e.dtype = dtype;
  e.sms = sms;
  const cudaError_t err = tg::launch_gated_grad(e, st);
  if (err != cudaSuccess) return fail_cuda("gated gradient launch", err);
  char* const sums = dgu + (two_terms(rows) ? 2 : 1) * o.dgu_bytes;
  char* const partials[2] = {sums, sums + o.plans.bytes[0]};
  return run_grads(o.p, o.plans, {dx_dev != nullptr, weights}, true, partials, sms, pairs, st);
}

int64_t tg_xent_fwd_workspace_bytes(int64_t rows, int64_t cols, int64_t vocab) {
  TG_TRY(check_xent(rows, cols, vocab, cols, cols, TG_BF16));
  if (rows == 0) return 0;
  int pairs = 0;
  TG_TRY(linear_ready(nullptr, &pairs));
  return static_cast<int64_t>(xent_fwd_plan({nullptr, rows, cols, cols, ""},
                                            {nullptr, vocab, cols, cols, ""}, {}, TG_BF16, pairs)
                                  .total);
}

int tg_xent_fwd(const void* x_dev, const void* w_dev, const int64_t* targets_dev, float* loss_dev,
                float* lse_dev, int64_t rows, int64_t cols, int64_t vocab, int64_t ld_x,
                int64_t ld_w, int64_t ignore_index, int dtype, void* workspace_dev,
                int64_t workspace_bytes, void* stream) {
  TG_TRY(check_xent(rows, cols, vocab, ld_x, ld_w, dtype));
  TG_TRY(check_workspace(nullptr, workspace_bytes, 0));
  if (rows == 0) return TG_OK;
  const Mat x = {x_dev, rows, cols, ld_x, "x"}, w = {w_dev, vocab, cols, ld_w, "w"};
  TG_TRY(check_array(loss_dev, 4, "loss"));
  TG_TRY(check_array(lse_dev, 4, "lse"));
  TG_TRY(check_mats({x, w}));
  TG_TRY(check_array(targets_dev, 8, "targets"));
  int sms = 0, pairs = 0;
  TG_TRY(linear_ready(&sms, &pairs));
  tg::XentRows loss = {};
  loss.targets = targets_dev;
  XentFwd o = xent_fwd_plan(x, w, loss, dtype, pairs);
  TG_TRY(check_workspace(workspace_dev, workspace_bytes, o.total));
  const uint64_t row4 = uint64_t(rows) * 4;
  const Region r[] = {{loss_dev, row4, "loss"}, {lse_dev, row4, "lse"},
                      {workspace_dev, o.total, "workspace"}, region(x), region(w),
                      {targets_dev, uint64_t(rows) * 8, "targets"}};
  TG_TRY(check_apart(r, 3, 6));
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  tg::XentJoin j = {};
  j.targets = targets_dev;
  j.ignore = ignore_index;
  j.loss = loss_dev;
  j.lse = lse_dev;
  j.rows = static_cast<uint32_t>(rows);
  j.vocab = static_cast<uint32_t>(vocab);
  cudaError_t e;
  if (o.logits.part_bytes) {
    char* const parts[1] = {static_cast<char*>(workspace_dev)};
    TG_TRY(run_products(&o.logits.p, &o.logits.plan, parts, 1, pairs, 0, -1, st));
    e = tg::launch_xent_rows(j, parts_of(o.logits.plan, parts[0]), st);
  } else {
    Product& p = o.logits.p;
    p.stats = workspace_dev;
    p.slots = o.slots;
    p.hit = reinterpret_cast<float*>(static_cast<char*>(workspace_dev) + o.stats_bytes);
    TG_TRY(whole_product(p, o.logits.plan, nullptr, sms, pairs, st));
    j.stats = p.stats;
    j.hit = p.hit;
    j.slots = o.slots;
    e = tg::launch_xent_join(j, st);
  }
  return e == cudaSuccess ? TG_OK : fail_cuda("cross entropy launch", e);
}

int64_t tg_xent_bwd_workspace_bytes(int64_t rows, int64_t cols, int64_t vocab) {
  TG_TRY(check_xent(rows, cols, vocab, cols, cols, TG_BF16));
  TG_TRY(check_tiles(vocab, cols));
  if (rows == 0) return 0;
  int pairs = 0;
  TG_TRY(linear_ready(nullptr, &pairs));
  return static_cast<int64_t>(xent_bwd_plan(rows, cols, vocab, TG_BF16, pairs).total);
}

int tg_xent_bwd(const float* dloss_dev, const void* x_dev, const void* w_dev,
                const int64_t* targets_dev, const float* lse_dev, void* dx_dev, void* dw_dev,
                int64_t rows, int64_t cols, int64_t vocab, int64_t ld_x, int64_t ld_w,
                int64_t ld_dx, int64_t ld_dw, int64_t ignore_index, int dtype,
                void* workspace_dev, int64_t workspace_bytes, void* stream) {
  TG_TRY(check_xent(rows, cols, vocab, ld_x, ld_w, dtype));
  TG_TRY(check_tiles(vocab, cols));
  if (dx_dev) TG_TRY(check_lds({{ld_dx, cols, "ld_dx"}}));
  if (dw_dev) TG_TRY(check_lds({{ld_dw, cols, "ld_dw"}}));
  TG_TRY(check_workspace(nullptr, workspace_bytes, 0));
  if (!dx_dev && !dw_dev) return TG_OK;
  const Mat x = {x_dev, rows, cols, ld_x, "x"}, w = {w_dev, vocab, cols, ld_w, "w"},
            dx = {dx_dev, dx_dev ? rows : 0, cols, ld_dx, "dx"},
            dw = {dw_dev, dw_dev ? vocab : 0, cols, ld_dw, "dw"};
  TG_TRY(check_mats({dx, dw}));
  if (rows > 0) {
    TG_TRY(check_mats({x, w}));
    TG_TRY(check_array(targets_dev, 8, "targets"));
    TG_TRY(check_array(dloss_dev, 4, "dloss"));
    TG_TRY(check_array(lse_dev, 4, "lse"));
  }
  int sms = 0, pairs = 0;
  TG_TRY(linear_ready(&sms, &pairs));
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (rows == 0) return zero_fill(dw, st);
  const XentBwd o = xent_bwd_plan(rows, cols, vocab, dtype, pairs);
  TG_TRY(check_workspace(workspace_dev, workspace_bytes, o.total));
  const uint64_t row4 = uint64_t(rows) * 4;
  const Region r[] = {region(dx), region(dw), {workspace_dev, o.total, "workspace"}, region(x),
                      region(w), {targets_dev, uint64_t(rows) * 8, "targets"},
                      {dloss_dev, row4, "dloss"}, {lse_dev, row4, "lse"}};
  TG_TRY(check_apart(r, 3, 8));
  char* base = static_cast<char*>(workspace_dev);
  char* const behind = base + (o.two ? 2 : 1) * o.dl_bytes;
  float* alpha = reinterpret_cast<float*>(behind);
  char* const parts[1] = {behind + kWorkspaceAlign};
  char* dx_sums = parts[0] + o.part_bytes;
  char* const partials[2] = {dx_sums, dx_sums + o.dx_bytes};
  const tg::XentRows loss = {dloss_dev, targets_dev, ignore_index, static_cast<uint32_t>(vocab), alpha};
  Product dx_first;
  Plan dx_plan = {};
  for (int64_t c = 0; c < o.chunks; ++c) {
    const int64_t first = c * o.chunk, n = vocab - first < o.chunk ? vocab - first : o.chunk;
    const Mat dl = {base, rows, n, o.chunk, "gradients of logits"};
    LogitsPlan logits =
        logits_plan(logits_product(tg::kEpiDlogits, x, w, first, n, loss, dtype), pairs);
    Product& p = logits.p;
    const Mat dl_rest = {base + o.dl_bytes, rows, n, o.chunk, "gradients of logits"};
    const Mat* rest = o.two ? &dl_rest : nullptr;
    if (logits.part_bytes) {
      TG_TRY(run_products(&p, &logits.plan, parts, 1, pairs, 0, -1, st));
      tg::XentDlogits d;
      d.loss = loss;
      d.lse = lse_dev;
      d.out = base;
      d.rows = static_cast<uint32_t>(rows);
      d.cols = static_cast<uint32_t>(n);
      d.first_col = static_cast<uint32_t>(first);
      d.pitch_out = static_cast<uint32_t>(o.chunk);
      d.dtype = dtype;
      d.sms = sms;
      const cudaError_t e = tg::launch_xent_dlogits(d, parts_of(logits.plan, parts[0]), st);
      if (e != cudaSuccess) return fail_cuda("cross entropy launch", e);
    } else {
      p.c[0] = dl;
      if (rest) p.c[1] = *rest;
      p.lse = lse_dev;
      TG_TRY(whole_product(p, logits.plan, nullptr, sms, pairs, st));
    }
    Product q[2] = {xent_dx_product(dl, rest, w, first, dx, dtype),
                    xent_dw_product(dl, rest, x, dw, first, dtype)};
    q[0].alpha = q[1].alpha = alpha;
    q[0].accumulate = !o.sums ? 0 : c == 0 ? 1 : 2;
    GradPlans plans(q, pairs, o.sums);
    if (c == 0)
      dx_first = q[0], dx_plan = plans.w[0];
    else if (plans.w[0].splits > dx_plan.splits)
      // each piece's sums have a place among the first one's
      plans.w[0] = plan_of(q[0], dx_plan.splits, true);
    TG_TRY(run_grads(q, plans, {dx_dev != nullptr, dw_dev != nullptr}, !o.sums, partials, sms, pairs, st));
  }
  char* const sums[1] = {dx_sums};
  return dx_dev && o.sums ? join_products(&dx_first, &dx_plan, sums, 1, sms, st) : TG_OK;
}

}  // extern "C"
