// Host build of the fused products' C ABI (tg_linear_api.cu with tg_api.cu) against a CUDA runtime and kernels
// that are not there, for the CPU tests: says what each call launches.
// usage: fused_ways_driver < calls, one "operator rows cols n" a line.  Prints a line of words for each.
#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdio>
#include <set>
#include <string>

#include "../include/tg.h"
#include "tg_few_config.h"
#include "tg_internal.h"
#include "tg_linear_config.h"

namespace {

constexpr int kPairs = 76;
std::set<std::string> words;
uint32_t first_splits;   // of the first piece of a vocabulary

const char* name_of(int epi) {
  const char* const names[] = {"store", "gated", "stats", "dlogits"};
  return names[epi];
}

CUresult encode(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                CUtensorMapL2promotion, CUtensorMapFloatOOBfill) {
  return CUDA_SUCCESS;
}

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
  for (int i = 0; i < l.products; ++i) {
    const LinearProduct& q = l.q[i];
    const std::string lies = q.a_mn ? "mn" : q.b_mn ? "kn" : "kk";
    const std::string way = std::string("pair-") + name_of(l.epi) + "-" + lies;
    words.insert(way);
    if (l.products == 2) words.insert(way + "-two");
    if (q.k_seg < q.k_blocks) words.insert(way + "-two-along-k");
    if (q.n_seg < q.n_blocks) words.insert(way + "-two-along-n");
    if (q.splits > 1) words.insert(way + "-split");
    if (q.split_from < q.m_blocks * q.n_blocks) words.insert(way + "-half-units");
    if (q.blocks_per_split > 8) words.insert(way + "-segments");
    if (q.partial == 1 && !q.a_mn) first_splits = q.splits;
    if (q.partial == 2) {
      words.insert(way + "-added");
      if (q.splits < first_splits) words.insert(way + "-added-fewer");
      if (q.splits > 1) words.insert(way + "-added-split");
    }
  }
  return cudaSuccess;
}
cudaError_t launch_few(const FewLaunch& l, cudaStream_t) {
  const std::string way = std::string("few-") + name_of(l.epi) + (l.w_mn ? "-kn" : "-kk");
  words.insert(way);
  words.insert(way + "-ranks" + std::to_string(l.ranks));
  words.insert(way + "-rows" + std::to_string(few_padded(l.rows)));
  if (l.groups > 1) words.insert(way + "-groups");
  if (l.terms == 2) words.insert(way + "-terms");
  if (l.k_seg < l.k_blocks) words.insert(way + "-two-along-k");
  return cudaSuccess;
}
cudaError_t launch_outer(const OuterLaunch& l, cudaStream_t) {
  words.insert("outer" + std::to_string(l.results));
  return cudaSuccess;
}
cudaError_t launch_linear_join(const LinearJoin*, int n, int, int, cudaStream_t) {
  words.insert("join" + std::to_string(n));
  return cudaSuccess;
}
cudaError_t launch_gated_join(const GatedJoin&, cudaStream_t) { return words.insert("gated-join"), cudaSuccess; }
cudaError_t launch_gated_grad(const GatedGrad&, cudaStream_t) { return cudaSuccess; }
cudaError_t launch_xent_join(const XentJoin&, cudaStream_t) { return words.insert("xent-join"), cudaSuccess; }
cudaError_t launch_xent_rows(const XentJoin&, const XentParts&, cudaStream_t) {
  return words.insert("xent-rows"), cudaSuccess;
}
cudaError_t launch_xent_dlogits(const XentDlogits&, const XentParts&, cudaStream_t) {
  return words.insert("xent-dlogits"), cudaSuccess;
}
}  // namespace tg

int main() {
  char op[32];
  long long r, c, n;
  // arrays far from one another, that nothing reads
  auto at = [](int i) { return reinterpret_cast<void*>((uintptr_t(i) + 1) << 42); };
  while (scanf("%31s %lld %lld %lld", op, &r, &c, &n) == 4) {
    words.clear();
    const std::string which = op;
    const int64_t big = int64_t(1) << 41;
    float* const f0 = static_cast<float*>(at(10));
    float* const f1 = static_cast<float*>(at(11));
    int64_t* const t = static_cast<int64_t*>(at(12));
    int rc = -1;
    if (which == "input_grad")
      rc = tg_input_grad(at(0), at(1), at(2), r, c, n, n, n, c, TG_F16, at(9), big, nullptr);
    else if (which == "gated_fwd")
      rc = tg_gated_fwd(at(0), at(1), at(2), at(3), at(4), at(5), r, c, n, c, n, n, n, n, n, TG_ACT_SILU,
                        TG_F16, at(9), big, nullptr);
    else if (which == "gated_bwd")
      rc = tg_gated_bwd(at(0), at(1), at(2), at(3), at(4), at(5), at(6), at(7), at(8), r, c, n, n, n, n, c, n,
                        n, c, n, n, TG_ACT_SILU, TG_F16, at(9), big, nullptr);
    else if (which == "xent_fwd")
      rc = tg_xent_fwd(at(0), at(1), t, f0, f1, r, c, n, c, c, -100, TG_F16, at(9), big, nullptr);
    else if (which == "xent_bwd")
      rc = tg_xent_bwd(f0, at(0), at(1), t, f1, at(2), at(3), r, c, n, c, c, c, c, -100, TG_F16, at(9), big,
                       nullptr);
    if (rc != 0) {
      printf("refused: %s\n", tg_last_error());
      return 1;
    }
    for (const std::string& w : words) printf("%s ", w.c_str());
    printf("\n");
  }
  return 0;
}
