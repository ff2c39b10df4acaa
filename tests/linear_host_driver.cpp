// Host build of the fused products' C ABI (tg_linear_api.cu with tg_api.cu) against a CUDA runtime and kernels
// that are not there, for the CPU tests: random calls of every entry point, with each tensor map and
// pointer that reaches a launch held against the buffers the call was given, and the units of every launch
// walked as the kernel walks them.
// usage: linear_host_driver seed calls.  Prints "ok calls launches few pairs2 splits groups parts pieces" or what
// is wrong.
#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <random>
#include <set>
#include <string>
#include <vector>

#include "../include/tg.h"
#include "tg_few_config.h"
#include "tg_internal.h"
#include "tg_tile_scheduler.cuh"

namespace {

constexpr int kPairs = 76;
struct Buffer {
  uintptr_t at;
  uint64_t bytes;
  std::string name;
};
std::vector<Buffer> buffers;
uintptr_t top;
long launches, few, two, splits, groups, parts, pieces;

[[noreturn]] void wrong(const std::string& what) {
  printf("wrong: %s\n", what.c_str());
  exit(1);
}

// A new buffer, far from the others.
void* buffer(uint64_t bytes, const char* name) {
  const uintptr_t at = top;
  top += (bytes + (1 << 20)) / 4096 * 4096 + 4096;
  buffers.push_back({at, bytes, name});
  return reinterpret_cast<void*>(at);
}

void inside(const void* p, uint64_t bytes, const char* what) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(p);
  for (const Buffer& b : buffers)
    if (a >= b.at && a + bytes <= b.at + b.bytes) return;
  wrong(std::string(what) + " reaches past its buffer");
}

// Tensor maps carry what they were encoded with in their first words.
struct Encoded {
  uint64_t base, inner, outer, pitch, elem;
};
CUresult encode(CUtensorMap* map, CUtensorMapDataType dt, cuuint32_t, void* base,
                const cuuint64_t* dims, const cuuint64_t* strides, const cuuint32_t* box,
                const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                CUtensorMapL2promotion, CUtensorMapFloatOOBfill) {
  const uint64_t elem = dt == CU_TENSOR_MAP_DATA_TYPE_FLOAT32 ? 4 : 2;
  const Encoded e = {reinterpret_cast<uint64_t>(base), dims[0], dims[1], strides[0], elem};
  memset(map, 0, sizeof(*map));
  memcpy(map, &e, sizeof(e));
  if (e.base % 16 || e.pitch % 16 || e.inner == 0 || e.outer == 0 || e.inner * elem > e.pitch ||
      box[0] * elem != 128 || box[1] > 256)
    return CUDA_ERROR_INVALID_VALUE;
  return CUDA_SUCCESS;
}

Encoded seen(const CUtensorMap& m, const char* what) {
  Encoded e;
  memcpy(&e, &m, sizeof(e));
  if (e.base == 0) wrong(std::string(what) + " was not encoded");
  inside(reinterpret_cast<void*>(e.base), (e.outer - 1) * e.pitch + e.inner * e.elem, what);
  return e;
}

// LinearUnits of tg_linear_kernel.cuh
void walk(const tg::LinearLaunch& l) {
  const uint32_t units[2] = {l.q[0].total_units * l.q[0].splits,
                             l.products == 2 ? l.q[1].total_units * l.q[1].splits : 0};
  const uint32_t step = l.grid / 2;
  std::set<std::pair<int, uint32_t>> done;
  for (uint32_t c = 0; c < step; ++c) {
    uint32_t at = c, which = 0, ahead = 0;
    const uint32_t busy = units[0] % step;
    auto rounds = [&]() { at = c + (busy ? (step - busy) * l.extra : 0); };
    auto second = [&]() {
      which = 1;
      if (l.extra && busy && c >= busy)
        ahead = l.extra, at = (c - busy) * l.extra;
      else
        rounds();
    };
    if (at >= units[0]) second();
    while (at < units[which]) {
      if (!done.insert({which, at}).second) wrong("a unit is walked twice");
      if (ahead > 1)
        --ahead, ++at;
      else if (ahead == 1)
        ahead = 0, rounds();
      else if ((at += step) >= units[0] && which == 0)
        second();
    }
  }
  if (done.size() != units[0] + units[1]) wrong("units are left out");
  for (int i = 0; i < l.products; ++i) {   // half units are the tiles after split_from
    const tg::LinearProduct& q = l.q[i];
    const uint32_t tiles = q.m_blocks * q.n_blocks;
    if (q.split_from + 2 * (tiles - q.split_from) != q.total_units || q.split_from > tiles)
      wrong("units and tiles");
    if (q.splits > 1 && q.total_units != tiles) wrong("split sums of half units");
    if ((q.splits - 1) * q.blocks_per_split >= q.k_blocks || q.splits * q.blocks_per_split < q.k_blocks)
      wrong("ranges of K");
  }
}

cudaError_t fine() { return cudaSuccess; }

}  // namespace

extern "C" {
cudaError_t cudaGetDevice(int* d) { return *d = 0, cudaSuccess; }
cudaError_t cudaGetLastError() { return cudaSuccess; }
const char* cudaGetErrorString(cudaError_t) { return "error"; }
const char* cudaGetErrorName(cudaError_t) { return "error"; }
cudaError_t cudaDeviceGetAttribute(int* v, cudaDeviceAttr a, int) {
  *v = a == cudaDevAttrComputeCapabilityMajor ? 10 : a == cudaDevAttrComputeCapabilityMinor ? 3 : 152;
  return cudaSuccess;
}
cudaError_t cudaPointerGetAttributes(cudaPointerAttributes* a, const void*) {
  a->type = cudaMemoryTypeDevice;
  a->device = 0;
  return cudaSuccess;
}
cudaError_t cudaGetDriverEntryPointByVersion(const char*, void** fn, unsigned int, unsigned long long,
                                             cudaDriverEntryPointQueryResult* r) {
  *fn = reinterpret_cast<void*>(&encode);
  *r = cudaDriverEntryPointSuccess;
  return cudaSuccess;
}
}

namespace tg {
cudaError_t prepare_gemm_kernels(int* pairs) { return *pairs = kPairs, cudaSuccess; }
cudaError_t prepare_linear_kernels(int* pairs) { return *pairs = kPairs, cudaSuccess; }

cudaError_t launch_linear(const LinearLaunch& l, cudaStream_t) {
  ++launches;
  two += l.products == 2;
  if (l.grid == 0 || l.grid % 2 || l.grid > 2 * kPairs) wrong("grid");
  for (int i = 0; i < l.products; ++i) {
    const LinearProduct& q = l.q[i];
    const bool two_k = q.k_seg < q.k_blocks, two_n = q.n_seg < q.n_blocks;
    const uint64_t k = uint64_t(q.k_seg) * kLinBK;
    for (int s = 0; s < (two_k ? 2 : 1); ++s) {
      const Encoded a = seen(q.a[s], "A");
      if ((q.a_mn ? a.inner : a.outer) != q.M || (q.a_mn ? a.outer : a.inner) > k) wrong("A's sizes");
      for (int n = 0; n < (two_n || l.epi == kEpiGated ? 2 : 1); ++n) {
        const Encoded b = seen(q.b[2 * s + n], "B");
        if ((q.b_mn ? b.inner : b.outer) != q.N) wrong("B's columns");
        if ((q.b_mn ? b.outer : b.inner) != (q.a_mn ? a.outer : a.inner)) wrong("K of A and B");
      }
    }
    splits += q.splits > 1;
    if (l.epi == kEpiStats) continue;
    for (int n = 0; n < (two_n ? 2 : 1); ++n) {
      const Encoded c = seen(q.c[n], "C");
      if (c.inner != q.N || c.elem != (q.partial ? 4u : 2u)) wrong("C's columns");
      if (q.partial ? c.outer != uint64_t(q.splits) * q.part_rows || q.part_rows % 32 || q.part_rows < q.M
                    : c.outer != q.M)
        wrong("C's rows");
    }
    if (q.splits > 1 && !q.partial) wrong("split sums without a place");
    if (q.alpha) inside(q.alpha, 4, "alpha");
  }
  if (l.epi == kEpiStats) {
    inside(l.stats, 8ull * l.q[0].M * l.slots, "statistics");
    inside(l.hit, 4ull * l.q[0].M, "targets' logits");
    if (l.slots < (l.q[0].N + kStatCols - 1) / kStatCols) wrong("slots");
  }
  if (l.epi == kEpiDlogits) inside(l.loss.alpha, 4, "alpha"), inside(l.lse, 4ull * l.q[0].M, "lse");
  if (l.epi == kEpiGated && l.keep) seen(l.q[0].c[1], "g"), seen(l.q[0].c[2], "u");
  walk(l);
  return fine();
}

cudaError_t launch_few(const FewLaunch& l, cudaStream_t) {
  ++few;
  groups += l.groups > 1;
  const bool gated = l.epi == kEpiGated, two_k = l.k_seg < l.k_blocks;
  for (int i = 0; i < (gated || two_k ? 2 : 1); ++i) {
    const Encoded w = seen(l.w[i], "weights"), x = seen(l.x[i], "rows");
    if ((l.w_mn ? w.inner : w.outer) != l.outs || x.outer != l.rows) wrong("few rows' sizes");
    if ((l.w_mn ? w.outer : w.inner) != x.inner || x.inner > uint64_t(l.k_seg) * kFewBK) wrong("K");
    if (l.terms == 2) seen(l.x_rest[i], "second term");
  }
  if (l.rows > uint32_t(kFewRows) || l.tiles * uint32_t(kFewM) < l.outs) wrong("few rows");
  if (l.ranks > 8 || (l.ranks & (l.ranks - 1)) || few_padded(l.rows) % l.ranks) wrong("cluster");
  const uint64_t row2 = 2ull * l.outs;
  if (l.partials)
    inside(l.partials, 4ull * l.groups * l.rows * l.outs, "groups' sums");
  else if (l.groups != 1)
    wrong("groups without a place");
  else if (l.epi == kEpiStats)
    inside(l.stats, 8ull * l.rows * l.slots, "statistics"), inside(l.hit, 4ull * l.rows, "logits");
  else
    inside(l.out, (l.rows - 1) * 2ull * l.ld_out + row2, "results");
  if (l.epi == kEpiStats && l.slots < l.tiles) wrong("slots");
  if (l.rest) inside(l.rest, (l.rows - 1) * 2ull * l.ld_out + row2, "second term");
  if (l.g) inside(l.g, (l.rows - 1) * 2ull * l.ld_g + row2, "g"), inside(l.u, (l.rows - 1) * 2ull * l.ld_u + row2, "u");
  return fine();
}

cudaError_t launch_outer(const OuterLaunch& l, cudaStream_t) {
  if (l.rows < 1 || l.rows > uint32_t(kTwoTermRows) || l.n % 8 || l.ld_b % 8) wrong("outer product");
  const uint64_t a = 2 * ((l.rows - 1) * l.ld_a + l.m), b = 2 * ((l.rows - 1) * l.ld_b + l.n);
  inside(l.a, a, "outer a");
  if (l.a_rest) inside(l.a_rest, a, "outer a's rest");
  for (int i = 0; i < l.results; ++i) {
    inside(l.b[i], b, "outer b");
    if (l.b_rest[i]) inside(l.b_rest[i], b, "outer b's rest");
    inside(l.out[i], 2 * ((uint64_t(l.m) - 1) * l.ld_out[i] + l.n), "outer results");
  }
  return fine();
}

cudaError_t launch_linear_join(const LinearJoin* j, int n, int, int, cudaStream_t) {
  if (n < 1 || n > 3) wrong("joins");
  for (int i = 0; i < n; ++i) {
    if (j[i].cols % 4) wrong("columns of a join");
    inside(j[i].partials, 4ull * (uint64_t(j[i].splits - 1) * j[i].part_rows + j[i].rows) * j[i].cols, "sums");
    inside(j[i].out, (j[i].rows - 1) * 2ull * j[i].ld_out + 2ull * j[i].cols, "joined results");
  }
  return fine();
}
cudaError_t launch_gated_join(const GatedJoin& j, cudaStream_t) {
  for (const float* p : {j.g_parts, j.u_parts})
    inside(p, 4ull * (uint64_t(j.splits - 1) * j.part_rows + j.rows) * j.outs, "sums of g, u");
  return fine();
}
cudaError_t launch_gated_grad(const GatedGrad& g, cudaStream_t) {
  inside(g.dgu, 4ull * g.rows * g.outs, "dg, du");
  if (g.rest) inside(g.rest, 4ull * g.rows * g.outs, "rest of dg, du");
  return fine();
}
cudaError_t launch_xent_join(const XentJoin&, cudaStream_t) { return fine(); }
cudaError_t launch_xent_rows(const XentJoin& j, const XentParts& p, cudaStream_t) {
  ++parts;
  inside(p.parts, 4ull * (uint64_t(p.splits - 1) * p.part_rows + j.rows) * p.pitch, "parts of logits");
  return fine();
}
cudaError_t launch_xent_dlogits(const XentDlogits& d, const XentParts& p, cudaStream_t) {
  ++parts;
  inside(p.parts, 4ull * (uint64_t(p.splits - 1) * p.part_rows + d.rows) * p.pitch, "parts of logits");
  if (d.pitch_out % 4) wrong("pitch");
  inside(d.out, 2ull * d.rows * d.pitch_out, "gradients of logits");
  return fine();
}
}  // namespace tg

int main(int argc, char** argv) {
  std::mt19937 rng(atoi(argv[1]));
  const int calls = atoi(argv[2]);
  auto size = [&](double lo, double hi) {
    const double u = rng() / 4294967296.0;
    return static_cast<int64_t>(lo * pow(hi / lo, u) + 0.5);
  };
  for (int i = 0; i < calls; ++i) {
    buffers.clear();
    top = 1ull << 32;
    const int64_t rows = size(1, i % 7 ? 9000 : 300000), cols = 8 * size(1, 1024), outs = 8 * size(1, 1024),
                  vocab = size(1, 140000);
    // strides with room between rows; the buffer ends with the last row
    auto pad = [&](int64_t n) { return (n + 7) / 8 * 8 + 8 * int64_t(rng() % 3); };
    auto mat = [&](int64_t r, int64_t c, int64_t ld, const char* name) {
      return buffer(2 * ((r - 1) * ld + c), name);
    };
    const int dtype = rng() % 2;
    const int64_t lc = pad(cols), lo = pad(outs), lw = pad(outs);
    int rc = 0;
    const int op = rng() % 5;
    const bool first = rng() % 4 != 0, second = !first || rng() % 4 != 0;
    auto workspace = [&](int64_t n) {
      if (n < 0) wrong(tg_last_error());
      return n ? buffer(n, "workspace") : nullptr;
    };
    if (op == 0) {
      const int64_t n = tg_input_grad_workspace_bytes(rows, cols, outs);
      rc = tg_input_grad(mat(rows, outs, lo, "dy"), mat(cols, outs, lw, "w"), mat(rows, cols, lc, "dx"), rows,
                         cols, outs, lo, lw, lc, dtype, workspace(n), n, nullptr);
    } else if (op == 1) {
      const int64_t n = tg_gated_fwd_workspace_bytes(rows, cols, outs);
      rc = tg_gated_fwd(mat(rows, cols, lc, "x"), mat(cols, outs, lw, "wg"), mat(cols, outs, lo, "wu"),
                        mat(rows, outs, lo, "h"), first ? mat(rows, outs, lw, "g") : nullptr,
                        first ? mat(rows, outs, lo, "u") : nullptr, rows, cols, outs, lc, lw, lo, lo, lw, lo,
                        0, dtype, workspace(n), n, nullptr);
    } else if (op == 2) {
      const int64_t n = tg_gated_bwd_workspace_bytes(rows, cols, outs);
      rc = tg_gated_bwd(mat(rows, outs, lo, "dh"), mat(rows, outs, lo, "g"), mat(rows, outs, lw, "u"),
                        mat(rows, cols, lc, "x"), mat(cols, outs, lw, "wg"), mat(cols, outs, lo, "wu"),
                        first ? mat(rows, cols, lc, "dx") : nullptr,
                        second ? mat(cols, outs, lo, "dwg") : nullptr,
                        second ? mat(cols, outs, lw, "dwu") : nullptr, rows, cols, outs, lo, lo, lw, lc, lw,
                        lo, lc, lo, lw, 1, dtype, workspace(n), n, nullptr);
    } else {
      float* loss = static_cast<float*>(buffer(4 * rows, "loss"));
      float* lse = static_cast<float*>(buffer(4 * rows, "lse"));
      int64_t* t = static_cast<int64_t*>(buffer(8 * rows, "targets"));
      if (op == 3) {
        const int64_t n = tg_xent_fwd_workspace_bytes(rows, cols, vocab);
        rc = tg_xent_fwd(mat(rows, cols, lc, "x"), mat(vocab, cols, lc, "w"), t, loss, lse, rows, cols, vocab,
                         lc, lc, -100, dtype, workspace(n), n, nullptr);
      } else {
        const int64_t n = tg_xent_bwd_workspace_bytes(rows, cols, vocab);
        const long before = launches + few;
        rc = tg_xent_bwd(loss, mat(rows, cols, lc, "x"), mat(vocab, cols, lc, "w"), t, lse,
                         first ? mat(rows, cols, lc, "dx") : nullptr,
                         second ? mat(vocab, cols, lc, "dw") : nullptr, rows, cols, vocab, lc, lc, lc, lc,
                         -100, dtype, workspace(n), n, nullptr);
        pieces += launches + few - before > 4;
      }
    }
    if (rc != 0) wrong(std::string("refused: ") + tg_last_error());
  }
  printf("ok %d %ld %ld %ld %ld %ld %ld %ld\n", calls, launches, few, two, splits, groups, parts, pieces);
  return 0;
}
