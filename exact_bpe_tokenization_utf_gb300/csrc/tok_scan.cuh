// Block-wide sums, and the halves of a cluster's barrier.
#pragma once
#include <cuda_runtime.h>

namespace tokgb {

// Exclusive sum of v over the block (blockDim.x a multiple of 32), and the
// total; sh holds blockDim.x / 32 words and may be reused once the call is over.
template <class T>
__device__ __forceinline__ T block_excl_sum(T v, T* total, T* sh) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
  T inc = v;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const T o = __shfl_up_sync(0xffffffffu, inc, off);
    if (lane >= off) inc += o;
  }
  if (lane == 31) sh[warp] = inc;
  __syncthreads();
  T pre = 0, tot = 0;
  for (int k = 0; k < nw; ++k) {
    const T x = sh[k];
    pre += k < warp ? x : T(0);
    tot += x;
  }
  *total = tot;
  __syncthreads();
  return pre + inc - v;
}

// The two halves of a cluster's barrier.  Only the first warp releases: what it
// wrote, and what the other warps wrote before a barrier of the CTA that lies
// between, is seen by the cluster; a release in each warp would wait for the
// warp's own stores, results that no other CTA reads among them.
__device__ __forceinline__ void cluster_arrive() {
  if (threadIdx.x < 32) asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  else asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
}
// without what anyone wrote: others' reads and their start are waited for
__device__ __forceinline__ void cluster_arrive_only() { asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

}  // namespace tokgb
