// Thread-block clusters: rank, barrier and reads of a peer's shared memory.
#pragma once

#include "sv_common.cuh"

namespace sv {

__device__ __forceinline__ unsigned cluster_rank() {
  unsigned r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
// The barrier in two halves: what a thread did before its arrival is seen behind every wait.
__device__ __forceinline__ void cluster_arrive() {
  __syncwarp();
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  __syncwarp();
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_sync() {
  cluster_arrive();
  cluster_wait();
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

__device__ __forceinline__ void remote_store(uint32_t a, float v) {
  asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(a), "f"(v) : "memory");
}
__device__ __forceinline__ void remote_store(uint32_t a, float4 v) {
  asm volatile("st.shared::cluster.v4.f32 [%0], {%1,%2,%3,%4};" ::"r"(a), "f"(v.x), "f"(v.y), "f"(v.z), "f"(v.w) : "memory");
}

// Join the partial results of a cluster's C CTAs (a power of two up to 8): acc [rows][stride] outputs
// against the maxima cm [rows] (log2 units), sums cl [rows].  The CTAs share the rows out;
// store(row, d4, x) takes four elements of a row.  weights: 8 floats per row that a CTA takes, of
// its own shared memory that no peer reads.  Every thread of every CTA calls it; no CTA returns
// before its shared memory has been read.  A remote read takes most of a microsecond, so that eight
// are always in flight: a thread's first outputs beside the maxima and sums (one unit of 64 rows in
// two CTAs took 5 us with reads one after another).
template <int D, typename Store>
__device__ __forceinline__ void cluster_merge(const float *acc, int stride, const float *cm, const float *cl, int rows,
                                              unsigned C, unsigned rank, float none, float *weights, Store &&store) {
  constexpr int S = 8, V = D / 4;
  cluster_sync();
  const int threads = (int)blockDim.x, tid = (int)threadIdx.x, shift = 31 - __clz((int)C);
  const int per = (rows + (int)C - 1) >> shift, r0 = (int)rank * per, n = (min(rows, r0 + per) - r0) * V;
  // slot k: element u + (k / C) threads of CTA k % C
  float4 y[S];
  auto fetch = [&](int u) {
#pragma unroll
    for (int k = 0; k < S; ++k) {
      const int at = u + (k >> shift) * threads;
      if (at < n)
        y[k] = remote_f32x4(remote_address(acc + (size_t)(r0 + at / V) * stride + 4 * (at % V), k & (C - 1)));
    }
  };
  fetch(tid);
  if (tid * V < n) {
    float w[S], sums[S], top = none, sum = 0.f;
#pragma unroll
    for (int c = 0; c < S; ++c) {
      w[c] = none;
      sums[c] = 0.f;
      if (c < (int)C) {
        w[c] = remote_f32(remote_address(cm + r0 + tid, c));
        sums[c] = remote_f32(remote_address(cl + r0 + tid, c));
      }
    }
#pragma unroll
    for (int c = 0; c < S; ++c) top = fmaxf(top, w[c]);
#pragma unroll
    for (int c = 0; c < S; ++c) {
      w[c] = exp2f(w[c] - top);
      sum = fmaf(w[c], sums[c], sum);
    }
    const float inv = sum > 0.f ? 1.f / sum : 0.f;
#pragma unroll
    for (int c = 0; c < S; ++c)
      if (c < (int)C) weights[tid * S + c] = w[c] * inv;
  }
  __syncthreads();
  const int step = (S >> shift) * threads;
  for (int u = tid; u < n; u += step) {
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int k = 0; k < S; ++k) {
      const int at = u + (k >> shift) * threads;
      if (at >= n) break;
      const float w = weights[at / V * S + (k & (C - 1))];
      x.x = fmaf(w, y[k].x, x.x);
      x.y = fmaf(w, y[k].y, x.y);
      x.z = fmaf(w, y[k].z, x.z);
      x.w = fmaf(w, y[k].w, x.w);
      if (((k + 1) & (C - 1)) == 0) {
        store(r0 + at / V, at % V, x);
        x = make_float4(0.f, 0.f, 0.f, 0.f);
      }
    }
    fetch(u + step);
  }
  cluster_sync();
}

}  // namespace sv
