// A launch into the time of the kernel in front of it.
#pragma once

#include <cuda_runtime.h>

namespace qs {

// A launch that may start before the kernel in front of it in the stream has ended (programmatic
// dependent launch); the kernel waits for that end itself, in every block.
template <typename... Params>
cudaError_t launch_behind(void (*kern)(Params...), dim3 grid, int threads, int smem,
                          cudaStream_t stream, Params... params) {
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid, cfg.blockDim = dim3(threads), cfg.dynamicSmemBytes = smem;
  cfg.stream = stream, cfg.attrs = &attr, cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, params...);
}

}  // namespace qs
