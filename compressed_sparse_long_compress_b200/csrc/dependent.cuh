// Programmatic dependent launch for the paged operators: their kernels follow one
// another (plan, write, attention) and are short, so the next one's blocks are set
// up while the last one drains.
#pragma once

#include "common.cuh"

namespace cslc {

// Waits until what precedes this kernel on its stream has finished and its writes
// are visible. First in every kernel launched by launch_after, before it touches
// memory that an earlier kernel may write or still read.
__device__ __forceinline__ void grid_dependency_wait() { asm volatile("griddepcontrol.wait;\n" ::: "memory"); }

// Launches `kernel` as a programmatic dependent of what precedes it on `stream`.
template <typename... P, typename... A>
cudaError_t launch_after(void (*kernel)(P...), dim3 grid, dim3 block, size_t smem, cudaStream_t stream, A&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...);
}

}  // namespace cslc
