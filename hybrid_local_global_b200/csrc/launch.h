// launch.h -- kernels that are brought up while the one before them still runs.
//
// launch_early() lets a kernel's CTAs start before the previous kernel of the
// stream has finished, if that one allowed it (let_next_start). Such a kernel
// calls after_previous() before it reads or writes anything that the previous
// one touches, and on every way out: the stream's next kernel waits for this
// one only.
#pragma once

#include <cuda_runtime.h>

namespace hlg {

__device__ __forceinline__ void let_next_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void after_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// cluster: CTAs of a cluster along x, 0 where the kernel declares it (or has none)
template <class... P, class... A>
cudaError_t launch_early(void (*kern)(P...), dim3 grid, int block, size_t smem, cudaStream_t st, int cluster,
                         const A&... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(block);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute at[2] = {};
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = cluster;
  at[1].val.clusterDim.y = 1;
  at[1].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = cluster > 0 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kern, args...);
}

}  // namespace hlg
