// Host side: the launch of a kernel that waits (ptx::grid_wait) before it
// touches memory, so that it may be set up while the grid before it in the
// stream drains (programmatic stream serialization).  It ends after everything
// it waited for.  Kernels without clusters that several CTAs share an SM with
// let their dependents be set up at once (ptx::launch_dependents); the rows'
// clusters do not: the next grid's, placed into what the first leaves, end up
// uneven (32 x 151936 log probabilities 8.3 against 6.6 us).
// Kernels back to back, by graph replay: 8 x 2560 x 2560 product 8.2 -> 5.5 us, 2048 x
// 4096 bf16 quantised 8.2 -> 6.6, one row's product onto 151936 tokens 64.8 -> 61.9;
// one row's log probabilities called from the host 11.3 -> 10.1.
#pragma once

#include <cuda_runtime.h>

namespace dspark {

template <typename... P, typename... A>
cudaError_t launch_overlapped(void (*kernel)(P...), unsigned grid, unsigned threads, unsigned smem, unsigned cluster,
                              cudaStream_t s, const A&... args) {
  cudaLaunchConfig_t c = {};
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = cluster;
  at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
  c.gridDim = dim3(grid);
  c.blockDim = dim3(threads);
  c.dynamicSmemBytes = smem;
  c.stream = s;
  c.attrs = at;
  c.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&c, kernel, P(args)...);
}

}  // namespace dspark
