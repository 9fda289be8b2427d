// launch.h -- kernel launches with programmatic dependent launch (PDL).
//
// A kernel launched with pdl = true may start while the previous kernel on the stream is
// still running: its CTAs run their set-up (barriers, TMEM, loads of the call's inputs) and then
// execute griddepcontrol.wait (grid_dep_wait in sm100.cuh), which returns once the previous
// grid has completed and its writes are visible.  Every kernel of a call therefore reads the
// outputs of the call's earlier kernels, and writes anything they read, only after
// grid_dep_wait.  Each kernel also signals griddepcontrol.launch_dependents early so that the
// next one can be scheduled.
// The first kernel of a decode, a prefill or a combination of partial states is launched plainly:
// it starts when all that was queued before the call is complete and visible.  The call's other
// kernels start after it has, so the inputs that they load ahead of their waits (lengths, block table,
// cache, weights) are complete too, whichever kernel, this library's or not, wrote them.  It costs
// nothing: the status word's memset in front of that kernel overlaps with no kernel either.
// The one-kernel calls of the paged cache wait before they read anything.
#pragma once

#include <cuda_runtime.h>

namespace hra {

template <typename... KArgs, typename... Args>
cudaError_t launch_kernel(void (*kern)(KArgs...), dim3 grid, dim3 block, size_t smem, cudaStream_t stream, bool pdl,
                          Args&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pdl ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kern, static_cast<KArgs>(args)...);
}

// The same with thread-block clusters of cluster_x CTAs along x (gridDim.x a multiple of it).
template <typename... KArgs, typename... Args>
cudaError_t launch_kernel_cluster(void (*kern)(KArgs...), dim3 grid, dim3 block, size_t smem, cudaStream_t stream,
                                  bool pdl, int cluster_x, Args&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = static_cast<unsigned>(cluster_x);
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pdl ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kern, static_cast<KArgs>(args)...);
}

}  // namespace hra
