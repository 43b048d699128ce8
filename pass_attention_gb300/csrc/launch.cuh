// Launches that overlap with the end of the kernel before them on the stream
// (programmatic dependent launch): the CTAs may start while that kernel's last
// ones run, and call wait_for_previous_kernel() before they touch anything that it
// reads or writes. Every CTA calls it, also one that has nothing to do: a kernel
// that ended without waiting would let the next one start before the one
// before it has ended. (begin_behind_waiting_kernel() is the exception.)
// Pointers of these kernels carry no __restrict__: it says that nobody else writes what they
// point to while the kernel runs, and lets the compiler move loads across the wait or through
// the path for data that does not change. Until the wait that is not so.
#pragma once

#include <cuda_runtime.h>

namespace oss {

// Returns when every kernel before this one on the stream has ended and its
// writes are visible.
__device__ __forceinline__ void wait_for_previous_kernel() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// For a kernel that reads nothing of the one before it, where every CTA of that one calls
// wait_for_previous_kernel() before let_next_kernel_start(): all that came earlier has
// ended when this one starts. (The fence keeps what an SM's L1 holds of older launches out.) A
// CTA of it still waits for the kernel before, at its end: the kernel behind this one
// waits for this one only.
__device__ __forceinline__ void begin_behind_waiting_kernel() { asm volatile("fence.acq_rel.gpu;" ::: "memory"); }

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
