// launch.cuh -- launches that may begin while the stream's previous kernel ends.
#pragma once

#include <cuda_runtime.h>

namespace qml {

// Launch with programmatic stream serialisation: the blocks may be scheduled
// when the previous kernel's last blocks exit, so the kernel calls
// after_previous() before its first access to memory that another kernel
// writes.  In a row of small
// kernels this hides most of a launch.  cluster: blocks of a cluster (1: none).
// The result is this launch's own: an error that another call left in the
// runtime (cudaGetLastError) is none of it.
template <class... P, class... A>
cudaError_t launch_after(void (*kernel)(P...), dim3 grid, unsigned threads, unsigned cluster, cudaStream_t s,
                         A&&... args) {
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = cluster, at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.stream = s;
  cfg.attrs = at;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...);
  if (e != cudaSuccess) cudaGetLastError();  // returned, not left behind for the thread's next call
  return e;
}

// Waits until the previous kernel of the stream has finished and its writes are
// visible (returns at once after an ordinary launch).
__device__ __forceinline__ void after_previous() { cudaGridDependencySynchronize(); }

// Lets the blocks of a following launch_after() kernel be scheduled before this
// one ends (once all its blocks have called this or exited).
__device__ __forceinline__ void let_next_start() { cudaTriggerProgrammaticLaunchCompletion(); }

}  // namespace qml
