// A kernel that adds up what the one before it left (programmatic dependent launch): its CTAs come onto the
// SMs as soon as the last CTAs of the one before have started, and wait there for its end.  The kernel before
// calls let_dependents(); the dependent one calls wait_for_previous() in every CTA before any return and before
// it reads anything that kernel wrote (what was there before that kernel may be read earlier).  Against plain
// launches, calls back to back: forward of 1024 tokens with its join 36.1 -> 33.3 us, one token against 64 long
// pasts 31.8 -> 29.5, layer norm backward of 655360 x 32 32.8 -> 29.8.
#pragma once

#include <cuda_runtime.h>

namespace lsrm {

__device__ __forceinline__ void let_dependents() { asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory"); }
__device__ __forceinline__ void wait_for_previous() { asm volatile("griddepcontrol.wait;\n" ::: "memory"); }

template <typename... K, typename... A>
inline bool launch_dependent(void (*kernel)(K...), dim3 grid, int threads, cudaStream_t s, A... args) {
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t c{};
  c.gridDim = grid;
  c.blockDim = dim3((unsigned)threads);
  c.stream = s;
  c.attrs = &attr;
  c.numAttrs = 1;
  return cudaLaunchKernelEx(&c, kernel, K(args)...) == cudaSuccess;
}

}  // namespace lsrm
