// The sliding-window instances of the tensor-core tree attention for paged caches, a translation
// unit of their own so that they compile beside the others.
#include "attention_tc_kernel.cuh"

namespace sv {

cudaError_t launch_tc_window_paged(const TcParams &p, int D, const TcPlan &pl, cudaStream_t s) {
  return launch_tc_plan<true, true>(p, D, pl, s);
}

}  // namespace sv
