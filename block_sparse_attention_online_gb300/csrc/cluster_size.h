// Clusters of sixteen CTAs are beyond what every device promises (eight): a part of one, or one
// whose groups of SMs have lost some, may have no room for them.  Host only.
#pragma once

#include <cuda_runtime_api.h>

namespace attn_skip {

constexpr int kLargeCluster = 16, kPortableCluster = 8;

// Allows `kernel` clusters of kLargeCluster and says whether there is room for one, with so much
// shared memory (which has to be allowed already).  Asked by every call, since the answer is the
// current context's: 0.4 us of host time.
inline bool large_cluster_fits(const void *kernel, int threads, size_t smem) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(kLargeCluster);
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = smem;
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeClusterDimension;
  at.val.clusterDim.x = kLargeCluster;
  at.val.clusterDim.y = at.val.clusterDim.z = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  int clusters = 0;
  const bool fits =
      cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) ==
          cudaSuccess &&
      cudaOccupancyMaxActiveClusters(&clusters, kernel, &cfg) == cudaSuccess && clusters > 0;
  if (!fits) (void)cudaGetLastError();  // (it is no error of the call's: eight will do)
  return fits;
}

}  // namespace attn_skip
