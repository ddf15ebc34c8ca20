// The sliding-window instances of the tensor-core tree attention for contiguous caches, a translation
// unit of their own so that they compile beside the others.
#include "attention_tc_kernel.cuh"

namespace sv {

cudaError_t launch_tc_window(const TcParams &p, int D, const TcPlan &pl, cudaStream_t s) {
  return launch_tc_plan<true, false>(p, D, pl, s);
}

}  // namespace sv
