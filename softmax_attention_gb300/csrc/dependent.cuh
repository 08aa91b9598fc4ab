// dependent.cuh -- kernels that start while the one before them in the stream still runs
// (programmatic dependent launch): their set-up, and the blocks of a grid that is nearly done, then
// have work beside them.
#pragma once

#include <cuda_runtime.h>

namespace fa {

// Waits until the kernel launched before this one has ended and its writes are visible.  (They are read by
// plain loads: read-only ones are for what no kernel writes while this one runs.)
__device__ __forceinline__ void wait_for_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// Lets the next kernel's blocks start as this grid's leave room, once every block has said so.
__device__ __forceinline__ void let_next_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// Launches `kernel` so that its blocks may start before the kernel ahead of it in the stream has ended.
template <typename... Params, typename... Args>
cudaError_t launch_dependent(void (*kernel)(Params...), unsigned grid_x, unsigned grid_y, unsigned threads, size_t shared,
                             cudaStream_t stream, const Args&... args) {
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t config{};
  config.gridDim = dim3(grid_x, grid_y);
  config.blockDim = dim3(threads);
  config.dynamicSmemBytes = shared;
  config.stream = stream;
  config.attrs = &attr;
  config.numAttrs = 1;
  return cudaLaunchKernelEx(&config, kernel, Params(args)...);
}

}  // namespace fa
