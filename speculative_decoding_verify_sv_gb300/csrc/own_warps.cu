// Whole prefixes, a warp per unit (warp_units.cuh): calls of sv_shared_attention with many short sequences.
#include "stacked_keys.cuh"
#include "warp_units.cuh"

namespace sv {

namespace {

template <int D, int NT>
__global__ void __launch_bounds__(kWinThreads, WarpLayout<D, NT, OwnKeys>::CTAS) own_warps_kernel(const __grid_constant__ OwnParams p) {
  warp_units<D, NT, OwnKeys>(p);
}

}  // namespace

cudaError_t launch_own_warps(OwnParams &p, int D, cudaStream_t s) {
  return launch_warps<OwnKeys>(p, D, s, [](auto d, auto nt) { return own_warps_kernel<d(), nt()>; });
}

}  // namespace sv
