// Host-side launch of the library's kernels with programmatic stream
// serialization (see griddep_wait in ptx.cuh): the next kernel's CTAs may be
// scheduled and run their set-up while this one finishes.
#pragma once

#include <cuda_runtime.h>

namespace nsk {

// Dynamic shared memory that a kernel with at most 8 KB of its own gets without
// asking: the default limit of 48 KB is on both together.
constexpr size_t SMEM_WITHOUT_ASKING = 40 * 1024;

template <typename P>
cudaError_t launch_pdl(void (*kern)(P), dim3 grid, dim3 block, size_t smem, cudaStream_t st, const P& p) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, p);
}

// The same in clusters of `cluster` CTAs along x (grid.x a multiple of it).
template <typename P>
cudaError_t launch_pdl_cluster(void (*kern)(P), dim3 grid, dim3 block, size_t smem, unsigned cluster, cudaStream_t st,
                               const P& p) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kern, p);
}

}  // namespace nsk
