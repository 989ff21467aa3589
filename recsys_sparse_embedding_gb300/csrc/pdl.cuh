// Programmatic dependent launch: a kernel launched this way may start while
// the stream's previous kernel still drains, so that its setup (barriers,
// tensor memory, descriptor fetches) costs no time of its own. It calls
// pdl_wait() before it touches global memory: that returns once every earlier
// kernel of the stream is complete and its writes are visible (the chain is
// complete because each kernel here waits). pdl_go() lets the next kernel
// start its own setup; it takes effect when every block has called it.
#pragma once
#include <cuda_runtime.h>

#include <utility>

namespace dsf {

__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void pdl_go() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// Whether a runtime call succeeded. The error of one that did not is taken out
// of the runtime's own record: an entry point that reads the record after its
// launches would answer for it.
inline bool succeeded(cudaError_t e) {
  if (e != cudaSuccess) (void)cudaGetLastError();
  return e == cudaSuccess;
}

template <class... P, class... A>
bool pdl_launch(void (*kernel)(P...), dim3 grid, unsigned block, cudaStream_t s, A&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(block);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return succeeded(cudaLaunchKernelEx(&cfg, kernel, std::forward<A>(args)...));
}

}  // namespace dsf
