// Tree attention over a sliding window with sinks for units of few query rows (sm_103a, bf16): the keys
// are a window's.  The kernel is unit_attention.cuh's.
#include "unit_attention.cuh"

namespace sv {

namespace {

template <int D, int NT, int RG>
__global__ void __launch_bounds__(kWinThreads, 2) window_attn_kernel(const __grid_constant__ WinParams p);

// The tree's nodes, the sinks before the window and the window.
struct WindowKeys {
  using Params = WinParams;
  static constexpr bool kWindow = true, kListed = false, kPieces = false;
  __device__ static __forceinline__ void begin(const Params &) { wait_previous(); }
  __device__ static __forceinline__ int sequence(const Params &, int bs) { return bs; }
  __device__ static __forceinline__ int first_node(const Params &, int) { return 0; }
  __device__ static __forceinline__ SharedPart shared_part(const Params &, int, bool, SharedPart *) {
    __syncthreads();
    return {};
  }
  template <int D, int NT, int RG>
  static auto kernel() {
    return window_attn_kernel<D, NT, RG>;
  }
};

template <int D, int NT, int RG>
__global__ void __launch_bounds__(kWinThreads, 2) window_attn_kernel(const __grid_constant__ WinParams p) {
  unit_attention<D, NT, RG, WindowKeys>(p);
}

}  // namespace

// The tensor-core kernel pads a unit's rows to 128 or 256 and pays more for a unit's start and
// for the launch, but takes long windows of many rows at twice the rate.  As fitted to measurements
// (us; D = 128, contiguous caches, 128 to 2048 units, 40 to 512 rows, windows 17 to 4097):
//   13 + units tiles / SMs (6 + 1.45 key tiles) + 2 SMs / units      (2.55 for 256 rows)
// e.g. 128 units of 104 rows: window 129 13 us here against 21, window 1025 36 against 33; 512 units
// of 64 rows: 24 against 39, 69 against 87; 8 units of 208 rows, window 4097: 20 against 85.
// Up to 32 rows this kernel runs at the memory's rate: 2048 units, window 1025: 172 against 270.
bool window_prefers_tc(int B, int N, int Hq, int Hkv, int span, int num_sms) {
  const int M = N * (Hq / Hkv);
  if (M <= 32) return false;
  const double units = (double)B * Hkv, sms = num_sms;
  const double here = window_plan((long long)B * Hkv, M, span / kWinGroup + N / kWinGroup + 2, num_sms).us;
  const double tiles = span / 128 + 2;
  const double there = 13 + units * ((M + 255) / 256) / sms * (6 + (M > 128 ? 2.55 : 1.45) * tiles) + 2 * sms / units;
  return there < here;
}

cudaError_t launch_window_attention(const AttnParams &a, int num_sms, cudaStream_t s) {
  WinParams p{};
  if (!unit_params(p, a, a.M)) return cudaErrorInvalidValue;
  const int span = a.window - 1 < a.cap ? a.window - 1 : a.cap;
  return launch_units<WindowKeys>(p, a.D, (long long)a.B * a.Hkv, span / kWinGroup + (a.N + a.sinks) / kWinGroup + 2, num_sms, s);
}

}  // namespace sv
