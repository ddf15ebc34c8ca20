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

}  // namespace

cudaError_t launch_listed_warps(ListedParams &p, int D, cudaStream_t s) {
  return launch_warps<ListedKeys>(p, D, s, [](auto d, auto nt) { return listed_warps_kernel<d(), nt()>; });
}
cudaError_t launch_joined_warps(PieceParams &p, int D, cudaStream_t s) {
  return launch_warps<JoinedKeys>(p, D, s, [](auto d, auto nt) { return joined_warps_kernel<d(), nt()>; });
}

}  // namespace sv
