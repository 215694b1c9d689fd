// Launches whose set-up overlaps the end of the kernel before them in the stream
// (programmatic stream serialization).  The kernel waits for that one's completion
// itself (await_previous_kernel), in all of its blocks and before anything else in
// global memory; with a plain kernel before it nothing changes.  The kernel before may
// still write while this one's blocks are there, so what it can have written (lengths,
// tables, slots, rows, queries, biases) is not read through the read-only path
// (__ldg, ld.global.nc), which is for memory that nobody writes during a kernel's life.
#pragma once

#include <cuda_runtime.h>

namespace ira {

template <typename K, typename P>
bool launch_dependent(K kern, dim3 grid, int threads, int smem, const P& prm, cudaStream_t stream,
                      unsigned cluster = 1) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kern, prm) == cudaSuccess && cudaGetLastError() == cudaSuccess;
}

}  // namespace ira
