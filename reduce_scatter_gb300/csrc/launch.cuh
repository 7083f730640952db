// launch.cuh -- launches of the layer kernels that overlap with the end of the
// kernel before them (programmatic dependent launch).
//
// A layer's calls follow one another on one stream, and many take only a few
// microseconds, as long as it takes to start a grid.  So each kernel lets the
// next one of these start as soon as its own blocks have started
// (begin_kernel), and waits for the one before it to be complete and its
// results visible before it touches memory that is not its own.  Every block
// waits before it does anything else or returns: a grid is then complete only
// after its predecessor is, and the order reaches back through any number of
// kernels.  After a kernel that does not take part, and before one, the
// stream's usual order holds.
#pragma once

#include <cuda_runtime.h>

#include "layer_common.h"

namespace dgl {

__device__ __forceinline__ void wait_for_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void let_next_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void begin_kernel() {
  let_next_start();
  wait_for_previous();
}

template <class... Params, class... Args>
int launch(void (*kernel)(Params...), dim3 grid, dim3 block, size_t smem, cudaStream_t stream, Args... args) {
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t c{};
  c.gridDim = grid;
  c.blockDim = block;
  c.dynamicSmemBytes = smem;
  c.stream = stream;
  c.attrs = &attr;
  c.numAttrs = 1;
  DGL_CUDA(cudaLaunchKernelEx(&c, kernel, Params(args)...));
  return DG_OK;
}

}  // namespace dgl
