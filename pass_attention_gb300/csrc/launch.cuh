// Launches that overlap with the end of the kernel before them on the stream
// (programmatic dependent launch): the CTAs may start while that kernel's last
// ones run, and call wait_for_previous_kernel() before they touch anything that it
// reads or writes. Every CTA calls it, also one that has nothing to do: a kernel
// that ended without waiting would let the next one start before the one
// before it has ended.
#pragma once

#include <cuda_runtime.h>

namespace oss {

// Returns when every kernel before this one on the stream has ended and its
// writes are visible.
__device__ __forceinline__ void wait_for_previous_kernel() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// The next kernel on the stream may be scheduled (it waits as above).
__device__ __forceinline__ void let_next_kernel_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

template <typename... Params, typename... Args>
cudaError_t launch_after(void (*kernel)(Params...), dim3 grid, int threads, int smem, cudaStream_t stream, Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

}  // namespace oss
