// Clusters of sixteen CTAs are beyond what every device promises (eight): a part of one, or one
// whose groups of SMs have lost some, may have no room for them.  Host only.
#pragma once

#include <cuda_runtime_api.h>

#include <atomic>

namespace attn_skip {

constexpr int kLargeCluster = 16, kPortableCluster = 8;

// What a kernel's callers have found out, by device: 0 not asked yet, 1 there is room, -1 not.
struct ClusterRoom {
  static constexpr int kDevices = 64;
  std::atomic<signed char> known[kDevices];
};

// Allows `kernel` clusters of kLargeCluster and says whether the current device has room for one.
// The device is asked once (with the most shared memory that a launch takes, which has to be
// allowed already).
inline bool large_cluster_fits(const void *kernel, int threads, size_t smem, ClusterRoom &room) {
  int device = 0;
  if (cudaGetDevice(&device) != cudaSuccess) return false;
  std::atomic<signed char> *known =
      device < ClusterRoom::kDevices ? &room.known[device] : nullptr;
  if (known)
    if (const signed char k = known->load(std::memory_order_relaxed)) return k > 0;
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
  if (known) known->store(fits ? 1 : -1, std::memory_order_relaxed);
  return fits;
}

}  // namespace attn_skip
