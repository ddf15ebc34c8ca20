// Whole prefixes, a CTA per unit (stacked_keys.cuh): calls of sv_shared_attention with little to read.
#include "stacked_keys.cuh"

namespace sv {

cudaError_t launch_own_units(OwnParams &p, int D, int groups, int num_sms, cudaStream_t s) {
  return launch_units<OwnKeys>(p, D, (long long)p.B * p.Hkv, groups, num_sms, s);
}

}  // namespace sv
