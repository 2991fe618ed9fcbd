// What the paged operators share: the reading of a page's scale, and programmatic
// dependent launch: their kernels follow one another (plan, write, attention) and
// are short, so the next one's blocks are set up while the last one drains.
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

// The exponent of a page's scale, which is a power of two: of any other number the largest one below it
// counts, held to the range of exponents that a scale may have.
constexpr int kScaleExpMin = -40, kScaleExpMax = 60;
__device__ __forceinline__ int page_scale_exponent(float scale) {
  return min(max((int)((__float_as_uint(scale) >> 23) & 0xffu) - 127, kScaleExpMin), kScaleExpMax);
}
__device__ __forceinline__ float pow2(int e) { return __uint_as_float((uint32_t)(127 + e) << 23); }   // e > -127

}  // namespace cslc
