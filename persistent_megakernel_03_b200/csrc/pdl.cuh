// pdl.cuh -- programmatic dependent launch: a kernel of an operator may be
// brought onto the SMs while the one before it in the stream still runs, and
// waits there for it.  It saves the launch gap (1 to 2 us of a 5 us operator).
//
// Every kernel launched this way waits (pdl_wait) in every CTA before it
// touches global memory that an earlier launch may write or read; weights,
// which none does, may be loaded before.  The wait returns when the launch
// before is complete and its writes are visible; as that launch waited for the
// one before it, all earlier work is complete too.  Such a kernel begins before
// its inputs are final: the operators on a decode's state read them with loads
// that L2 answers (__ldcg, cp.async.cg), never through the read-only path.  In
// a normal launch both calls do nothing.
#pragma once
#include <cuda_runtime.h>

namespace mk {

__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
// Lets the next launch of the stream begin once every CTA is past this point.
__device__ __forceinline__ void pdl_trigger() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// `cluster` CTAs (along x) share their shared memory.
template <typename... P, typename... A>
cudaError_t pdl_launch_cluster(void (*kernel)(P...), dim3 grid, dim3 block, int cluster, cudaStream_t st, A... args) {
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...);
}

template <typename... P, typename... A>
cudaError_t pdl_launch(void (*kernel)(P...), dim3 grid, dim3 block, size_t smem, cudaStream_t st, A... args) {
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...);
}

}  // namespace mk
