// The own keys behind shared ones, a CTA per unit (stacked_keys.cuh).
#include "stacked_keys.cuh"

namespace sv {

cudaError_t launch_joined_units(PieceParams &p, int D, int num_sms, cudaStream_t s) {
  // (the plan's forms go by some hundred own keys)
  return launch_units<JoinedKeys>(p, D, (long long)p.B * p.Hkv, p.N / kWinGroup + 18, num_sms, s);
}

}  // namespace sv
