// launch.cuh — launching a kernel under the end of the one before it.
#pragma once

#include <cstdint>
#include <type_traits>

#include <cuda_runtime.h>

namespace smla {

// Launch a kernel that waits for the one before it on the stream by itself
// (griddepcontrol.wait), so that its launch and setup pass under that one's end:
// 1 to 2 us of a call, 3 of the windowed attention's merge.
template <class Params>
cudaError_t launch_early(void (*kernel)(Params), unsigned ctas, int threads, uint32_t smem,
                         cudaStream_t stream, const std::remove_const_t<Params>& p) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

}  // namespace smla
