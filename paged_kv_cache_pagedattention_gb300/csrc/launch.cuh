// Kernels whose blocks come up while the kernel before them in the stream ends.
#pragma once

#include <cuda_runtime.h>

namespace pa {

// The kernel before this one in the stream has ended, and what it wrote is there.  A kernel that
// is launched by launch_early calls this before it reads or writes any memory but its own.
__device__ __forceinline__ void previous_done() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// The kernel behind this one in the stream, if launched by launch_early, may come up as soon as
// all blocks of this one have.  For a call's own second kernel: between calls it gained nothing
// and its waiting blocks stood in the way (long forks, captured, 25 -> 30 us).
__device__ __forceinline__ void next_may_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// A launch that may begin when the kernel before it ends, without a gap for the end to be seen
// by the host's queue.  Eager calls back to back on inputs that change from call to call, without
// and with it: beam selection of one request 12.3 and 8.1 us, of 128 rows of 131,072 bf16 24.6 and
// 19.4 (its join included), the rotary write of 2,176 tokens 15.5 and 13.1, fork, append, copy and
// release of long forks 34.0 and 28.1.  Clusters of `cluster` blocks along x.
template <typename P>
cudaError_t launch_early(void (*kernel)(P), dim3 grid, int threads, size_t smem, int cluster, const P& p,
                         cudaStream_t stream) {
  cudaLaunchConfig_t config = {};
  config.gridDim = grid;
  config.blockDim = dim3(threads);
  config.dynamicSmemBytes = smem;
  config.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  config.attrs = attr;
  config.numAttrs = cluster > 1 ? 2 : 1;
  const cudaError_t e = cudaLaunchKernelEx(&config, kernel, p);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace pa
