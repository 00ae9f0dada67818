// launch.cuh - launches that overlap their start with the end of the kernel
// before them in the stream (programmatic dependent launch).
//
// A kernel launched by after() may be placed while its predecessor still
// runs, once every CTA of that one has called begin() or ended; it calls
// begin() before it touches memory, which waits until the predecessor has
// ended and its writes are visible, so the order of effects in the stream is
// the usual one.  Every thread of every CTA calls it, so that a kernel's end
// implies its predecessor's.  Calls behind one another: the decode of one
// short context 12.3 -> 9.4 us, a batch's append 6.1 -> 4.1 us.
#pragma once

#include <cuda_runtime.h>

namespace nats {

__device__ __forceinline__ void begin() {
  cudaGridDependencySynchronize();
  cudaTriggerProgrammaticLaunchCompletion();
}

template <class... P, class... A>
cudaError_t after(void (*kernel)(P...), unsigned grid, dim3 block, size_t smem, cudaStream_t st, unsigned cluster,
                  A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim = {cluster, 1, 1};
  cfg.attrs = at;
  cfg.numAttrs = cluster > 0 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

}  // namespace nats
