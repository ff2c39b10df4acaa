// Host build of the C ABI (tg_api.cu, tg_train_api.cu) against a CUDA runtime and kernels that are not
// there, for the CPU tests: what a weight gradient would launch, and what the GEMM makes of the device.
// usage: train_host_driver gemm_pairs wgrad_pairs rows cols outs scale_offset
// (wgrad_pairs < 0: its kernels cannot be set up).  Prints
//   "gemm rc workers" of a pair launch at 8192^3, "setup n" (weight-gradient set-ups so far), then
//   "wgrad rc halves splits blocks_per_split k_blocks split_from units grid tma_scales workspace setup".
#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdio>
#include <cstdlib>

#include "../include/tg.h"
#include "tg_internal.h"

namespace {
int gemm_pairs, wgrad_pairs, setups;
tg::WgradLaunch launched;

CUresult encode(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill) {
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
cudaError_t prepare_gemm_kernels(int* pairs) { return *pairs = gemm_pairs, cudaSuccess; }
cudaError_t prepare_wgrad_kernels(int* pairs) {
  ++setups;
  *pairs = wgrad_pairs;
  return wgrad_pairs < 0 ? cudaErrorInvalidValue : cudaSuccess;
}
cudaError_t launch_wgrad(int, bool, const WgradLaunch& l, cudaStream_t) {
  launched = l;
  return cudaSuccess;
}
}  // namespace tg

int main(int argc, char** argv) {
  if (argc != 7) return 2;
  gemm_pairs = std::atoi(argv[1]);
  wgrad_pairs = std::atoi(argv[2]);
  const long rows = std::atol(argv[3]), cols = std::atol(argv[4]), outs = std::atol(argv[5]);
  int workers = 0;
  int rc = tg_gemm_launch_shape(8192, 8192, 8192, TG_VARIANT_PAIR, nullptr, nullptr, nullptr, nullptr,
                                nullptr, &workers, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr,
                                nullptr);
  std::printf("gemm %d %d\nsetup %d\n", rc, workers, setups);
  const uintptr_t gib = uintptr_t(1) << 40;   // regions far apart, never touched
  auto at = [&](int i, long off) { return reinterpret_cast<char*>((i + 1) * gib + off); };
  const int64_t bytes = tg_ckpt8_wgrad_workspace_bytes(rows, cols, outs);
  rc = bytes < 0 ? static_cast<int>(bytes)
                 : tg_ckpt8_wgrad(at(0, 0), at(1, std::atol(argv[6])), at(2, 0), at(3, 0), rows, cols,
                                  outs, outs, outs, TG_BF16, at(4, 0), bytes, nullptr);
  const tg::WgradLaunch& l = launched;
  std::printf("wgrad %d %u %u %u %u %u %u %u %u %lld %d\n", rc, l.halves, l.splits, l.blocks_per_split,
              l.k_blocks, l.split_from, l.total_units, l.grid, l.tma_scales,
              static_cast<long long>(bytes), setups);
  return 0;
}
