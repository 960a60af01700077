// dependent_launch.cuh -- launches that overlap their set-up with the end of
// the kernel before them in the stream (programmatic dependent launch).  The
// serving kernels take a few microseconds each and follow one another, so
// that a launch's own latency (about 1 us) is worth hiding.
#pragma once

#include <cuda_runtime.h>

namespace splash {

// First statement of such a kernel, before it reads or writes any memory:
// waits until everything before it in the stream has completed, and lets the
// next kernel's blocks be placed (they wait here in turn).  What follows reads
// global memory with ordinary loads: the kernel before may have written it
// while this one was already resident, so that it is not constant for this
// kernel's lifetime (ld.global.nc may be moved above the wait).
__device__ __forceinline__ void grid_dependency() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// cluster: CTAs per thread-block cluster (along x), 1: none.
template <class... Params, class... Args>
cudaError_t launch_dependent(void (*kernel)(Params...), dim3 grid, dim3 block, size_t smem, int cluster,
                             cudaStream_t stream, const Args &...args) {
  cudaLaunchConfig_t config = {};
  config.gridDim = grid;
  config.blockDim = block;
  config.dynamicSmemBytes = smem;
  config.stream = stream;
  cudaLaunchAttribute attrs[2] = {};
  attrs[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attrs[0].val.programmaticStreamSerializationAllowed = 1;
  attrs[1].id = cudaLaunchAttributeClusterDimension;
  attrs[1].val.clusterDim.x = (unsigned)cluster;
  attrs[1].val.clusterDim.y = attrs[1].val.clusterDim.z = 1;
  config.attrs = attrs;
  config.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&config, kernel, static_cast<Params>(args)...);
}

}  // namespace splash
