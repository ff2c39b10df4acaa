// tg_launch.cuh -- kernel launch with programmatic stream serialization, for every translation
// unit that holds kernels.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>
#include <utility>

namespace tg {

// Launches ``kernel`` with programmatic stream serialization: it may be scheduled while the
// previous kernel in the stream is still finishing (as that kernel's CTAs exit).  Every kernel
// launched this way issues griddepcontrol.wait before its first global memory access, so the
// stream's ordering of memory effects is unchanged; what overlaps is the launch itself and each
// CTA's set-up (barriers, TMEM allocation, descriptor prefetch).
template <typename... KArgs, typename... Args>
cudaError_t launch_pdl(void (*kernel)(KArgs...), dim3 grid, uint32_t threads, size_t smem,
                       cudaStream_t stream, Args&&... args) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, std::forward<Args>(args)...);
}

}  // namespace tg
