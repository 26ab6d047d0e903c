// The start of a cluster's CTAs: their shared memory may be written once every one of
// them has begun.  The arrival comes first in a kernel and the wait before the first
// remote write, so that what lies between hides it.  Whole warps.
#pragma once

namespace attn_skip {
namespace {

__device__ __forceinline__ void cluster_started() {
  asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

}  // namespace
}  // namespace attn_skip
