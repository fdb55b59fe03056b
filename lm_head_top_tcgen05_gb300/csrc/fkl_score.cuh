// What the scoring operators share: the given tokens, whose ids are 32 or 64 bits wide, and clusters of CTAs.
#pragma once

#include <cstdint>

namespace fkl {

struct TokenIds {
  const void* p;
  int32_t bytes;  // 4 or 8
  // The token at `at`, or -1 where it is outside [0, V).
  __device__ __forceinline__ int get(int64_t at, int V) const {
    const int64_t v = bytes == 8 ? static_cast<const int64_t*>(p)[at] : static_cast<const int32_t*>(p)[at];
    return v >= 0 && v < V ? static_cast<int>(v) : -1;
  }
};

// The same place of shared memory in the cluster's CTA `rank`.
template <class P>
__device__ __forceinline__ P* peer(P* p, int rank) {
  uint64_t a;
  asm volatile("mapa.u64 %0, %1, %2;" : "=l"(a) : "l"(reinterpret_cast<uint64_t>(p)), "r"(rank));
  return reinterpret_cast<P*>(a);
}
__device__ __forceinline__ int cluster_size() {
  uint32_t n;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(n));
  return static_cast<int>(n);
}
// The two halves of the cluster's barrier: shared memory written before `arrive` is seen by every CTA after `wait`.
__device__ __forceinline__ void cluster_arrive() {
  __syncwarp();
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  __syncwarp();
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
}  // namespace fkl
