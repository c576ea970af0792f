// Dependent launches: a kernel's start overlaps the end of the one ahead of it.
#pragma once

#include <cuda_runtime.h>

namespace fa {

// A kernel launched as dependent (launch_dependent) may start before the one
// ahead of it in the stream is done: it waits here, before it reads anything of that one's,
// until that one is complete and its writes are visible.
__device__ __forceinline__ void wait_for_previous_kernel() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
// Lets the next kernel start as soon as every CTA of this one has got here.
__device__ __forceinline__ void let_next_kernel_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// Launches `kernel` as dependent on the kernel ahead of it in the stream: its launch
// overlaps that one's end (a few microseconds less between them).  The kernel has to call
// wait_for_previous_kernel() before it reads what that one writes.
template <class... P, class... A>
cudaError_t launch_dependent(void (*kernel)(P...), dim3 grid, dim3 block, size_t smem, cudaStream_t stream, const A&... args) {
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, P(args)...);
}

}  // namespace fa
