// State of the current device that entry points outside attn_api.cu need.
#pragma once
#include <cstdint>
#include <utility>

#include <cuda_runtime.h>

namespace gb300 {

// SM count and the device status word (first failure recorded by a kernel) of the current device, and the id of its
// context (0 if that cannot be read), unless context is null. False, with nothing written, when the device cannot be
// queried.
bool device_state(int* num_sms, uint32_t** status, unsigned long long* context = nullptr);

// Launches a kernel as a programmatic dependent: its CTAs may be scheduled while the kernel before still runs, so every
// one of its threads begins with griddep_wait(), which returns when that kernel has ended and its writes can be seen.
template <class... P, class... A>
cudaError_t launch_dependent(void (*kernel)(P...), dim3 grid, dim3 block, size_t smem, cudaStream_t stream, A&&... args) {
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, std::forward<A>(args)...);
}

}  // namespace gb300
