// Listed pages, and the own keys behind shared ones, a warp per unit (warp_units.cuh).
#include "stacked_keys.cuh"
#include "warp_units.cuh"

namespace sv {

namespace {

template <int D, int NT>
__global__ void __launch_bounds__(kWinThreads, WarpLayout<D, NT, ListedKeys>::CTAS) listed_warps_kernel(const __grid_constant__ ListedParams p) {
  warp_units<D, NT, ListedKeys>(p);
}
template <int D, int NT>
__global__ void __launch_bounds__(kWinThreads, WarpLayout<D, NT, JoinedKeys>::CTAS) joined_warps_kernel(const __grid_constant__ PieceParams p) {
  warp_units<D, NT, JoinedKeys>(p);
}

template <int D, int NT, class Keys, class P>
cudaError_t launch_typed(void (*kern)(P), const P &p, cudaStream_t s) {
  constexpr int smem = WarpLayout<D, NT, Keys>::SMEM;
  static std::atomic<bool> attr[64];
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev < 0 || dev >= 64 || !attr[dev].load()) {
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < 64) attr[dev].store(true);
  }
  return launch_close(kern, dim3(((unsigned)p.units + 3) / 4), kWinThreads, (size_t)smem, s, p);
}

// 8-column steps of a unit's rows
template <class P>
int steps(const P &p) {
  return ((p.M + p.m_tiles - 1) / p.m_tiles + 7) / 8;
}

template <int D>
cudaError_t launch_listed(const ListedParams &p, cudaStream_t s) {
  switch (steps(p)) {
    case 1: return launch_typed<D, 1, ListedKeys>(listed_warps_kernel<D, 1>, p, s);
    case 2: return launch_typed<D, 2, ListedKeys>(listed_warps_kernel<D, 2>, p, s);
    case 3: return launch_typed<D, 3, ListedKeys>(listed_warps_kernel<D, 3>, p, s);
    default: return launch_typed<D, 4, ListedKeys>(listed_warps_kernel<D, 4>, p, s);
  }
}
template <int D>
cudaError_t launch_joined(const PieceParams &p, cudaStream_t s) {
  switch (steps(p)) {
    case 1: return launch_typed<D, 1, JoinedKeys>(joined_warps_kernel<D, 1>, p, s);
    case 2: return launch_typed<D, 2, JoinedKeys>(joined_warps_kernel<D, 2>, p, s);
    case 3: return launch_typed<D, 3, JoinedKeys>(joined_warps_kernel<D, 3>, p, s);
    default: return launch_typed<D, 4, JoinedKeys>(joined_warps_kernel<D, 4>, p, s);
  }
}

}  // namespace

cudaError_t launch_listed_warps(ListedParams &p, int D, cudaStream_t s) { return D == 128 ? launch_listed<128>(p, s) : launch_listed<64>(p, s); }
cudaError_t launch_joined_warps(PieceParams &p, int D, cudaStream_t s) { return D == 128 ? launch_joined<128>(p, s) : launch_joined<64>(p, s); }

}  // namespace sv
