// Thread-block clusters: rank, barrier and reads of a peer's shared memory.
#pragma once

#include "sv_common.cuh"

namespace sv {

__device__ __forceinline__ unsigned cluster_rank() {
  unsigned r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n"
               "barrier.cluster.wait.acquire.aligned;\n" ::: "memory");
}
// The address of a shared-memory variable in CTA `rank` of this cluster, and reads there.
__device__ __forceinline__ uint32_t remote_address(const void *local, unsigned rank) {
  uint32_t a;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(local)), "r"(rank));
  return a;
}
__device__ __forceinline__ float remote_f32(uint32_t a) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ float4 remote_f32x4(uint32_t a) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(a)
               : "memory");
  return v;
}

// Join the partial results of a cluster's CTAs: acc [rows][stride] outputs against the maxima
// cm [rows] (log2 units), sums cl [rows].  The CTAs share the rows out; store(row, d4, x, 1 / sum)
// takes four elements of a row.  Every thread of every CTA calls it; no CTA returns before its
// shared memory has been read.
template <int D, typename Store>
__device__ __forceinline__ void cluster_merge(const float *acc, int stride, const float *cm, const float *cl, int rows,
                                              unsigned C, unsigned rank, float none, Store &&store) {
  cluster_sync();
  const int threads = (int)blockDim.x;
  for (int u = (int)rank * threads + (int)threadIdx.x; u < rows * (D / 4); u += (int)C * threads) {
    const int r = u / (D / 4), d4 = u % (D / 4);
    float top = none;
    for (unsigned c = 0; c < C; ++c) top = fmaxf(top, remote_f32(remote_address(cm + r, c)));
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
    float sum = 0.f;
    for (unsigned c = 0; c < C; ++c) {
      const float w = exp2f(remote_f32(remote_address(cm + r, c)) - top);
      const float4 y = remote_f32x4(remote_address(acc + (size_t)r * stride + 4 * d4, c));
      sum += w * remote_f32(remote_address(cl + r, c));
      x.x += w * y.x;
      x.y += w * y.y;
      x.z += w * y.z;
      x.w += w * y.w;
    }
    store(r, d4, x, sum > 0.f ? 1.f / sum : 0.f);
  }
  cluster_sync();
}

}  // namespace sv
