// The own keys behind shared ones, a CTA per unit (stacked_keys.cuh).
#include "stacked_keys.cuh"

namespace sv {

cudaError_t launch_joined_units(PieceParams &p, int D, int groups, int num_sms, cudaStream_t s) {
  return launch_units<JoinedKeys>(p, D, (long long)p.B * p.Hkv, groups, num_sms, s);
}

}  // namespace sv
