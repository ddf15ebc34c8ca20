// Listed pages, a CTA per unit (stacked_keys.cuh).
#include "stacked_keys.cuh"

namespace sv {

cudaError_t launch_listed_units(ListedParams &p, int D, int groups, int num_sms, cudaStream_t s) {
  return launch_units<ListedKeys>(p, D, (long long)p.B * p.sets * p.Hkv, groups, num_sms, s);
}

}  // namespace sv
