// Two kernels of one call: the second may start before the first is done.
#pragma once

#include <cuda_runtime.h>

namespace fp8kv {

// A kernel whose launch attribute lets it start while the one before it in the stream still runs:
// nothing of that one's may be read above this line.  The other side lets it start.
__device__ __forceinline__ void wait_for_previous_kernel() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void let_next_kernel_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// For CTAs of the second kernel that have nothing to do: one of them waits all the same, so that the kernel
// is not done, and whatever follows it in the stream does not start, before the first one is.
__device__ __forceinline__ void leave_in_order() {
  if (blockIdx.x == 0 && blockIdx.y == 0 && blockIdx.z == 0) wait_for_previous_kernel();
}

// Launch with that attribute.
template <class... A>
cudaError_t launch_dependent(void (*fn)(A...), dim3 grid, int threads, int smem, cudaStream_t st, const A&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, fn, args...);
}

}  // namespace fp8kv
