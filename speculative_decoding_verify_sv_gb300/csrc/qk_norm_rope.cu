// Per-head norms of queries and keys with the position rotation, in one pass (sm_103a).
//
// A token's projection row holds Hq query heads, Hkv key heads and Hkv value heads of D
// elements.  Each query and key head x becomes
//   y = x / sqrt(mean(x^2) + eps) * w,
// and then the pairs (a, b) of its first `rot` elements turn by the angle position * inv_freq_i:
//   (a cos - b sin, a sin + b cos),
// the pairs being (i, i + rot/2), or neighbours (2i, 2i + 1).  Values are copied.  Everything
// between the load and the one rounding at the store is in fp32.
//
// Angles: a position is a whole number, so only the fraction of a turn per position matters.
// It is held as a 64-bit fixed-point fraction (of 2^64), which the 64-bit product with the
// position wraps exactly: no argument reduction and no loss at far positions (the error is
// that of the frequency, 2^-53 of it per position).  The nearest quarter turn comes off in
// integers, so that the sine and cosine are taken of at most an eighth of a turn.
//
// A warp takes a token (or, when there are few tokens, a part of its heads), reads whole heads
// with 16-byte loads, several in flight per lane, and computes the token's rot/2 sines and
// cosines once for all its heads.  It is bound by HBM: each element is read once and written
// once.
#include "sv_common.cuh"
#include "sv_internal.h"

namespace sv {

namespace {

constexpr int kRopeWarps = 8;
constexpr int kRopeUnroll = 4;  // 16-byte loads in flight per lane

template <typename T>
__device__ __forceinline__ uint4 pack_vec(const float *f);
template <>
__device__ __forceinline__ uint4 pack_vec<bf16>(const float *f) {
  return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7]));
}
template <>
__device__ __forceinline__ uint4 pack_vec<float>(const float *f) {
  return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
}

// The fraction of a turn per position, of 2^64.
__device__ __forceinline__ uint64_t turn_fraction(double inv_freq) {
  const double turns = inv_freq * 0.15915494309189533577;  // 1 / (2 pi)
  return __double2ull_rn((turns - floor(turns)) * 18446744073709551616.0);
}

// (cos, sin) of position * frequency.
__device__ __forceinline__ float2 turn_cos_sin(uint64_t fraction, long long position) {
  const uint64_t x = fraction * (uint64_t)position;         // of 2^64, wrapped to one turn
  const uint64_t quarter = (x + (1ull << 61)) >> 62;        // nearest quarter turn (4 = 0)
  const long long rest = (long long)(x - (quarter << 62));  // at most 2^61: an eighth of a turn
  float s, c;
  sincospif((float)rest * 1.0842021724855044e-19f, &s, &c);  // 2^-63: in half turns
  const float cq = (quarter & 1) ? -s : c, sq = (quarter & 1) ? c : s;
  return (quarter & 2) ? make_float2(-cq, -sq) : make_float2(cq, sq);
}

// LPH lanes hold one head of D = LPH * 16 / sizeof(T) elements, 16 bytes each.
template <typename T, int LPH, bool INTERLEAVED>
__global__ void __launch_bounds__(kRopeWarps * 32) qk_norm_rope_kernel(const __grid_constant__ RopeParams p) {
  constexpr int V = Elem<T>::kVec;
  constexpr int D = LPH * V, HPW = 32 / LPH;  // heads per warp-wide load
  __shared__ __align__(16) float2 s_cs[kRopeWarps][64];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int l = lane % LPH, sub = lane / LPH, e0 = l * V;
  const int half = p.rot >> 1, H = p.Hq + 2 * p.Hkv;
  const bool turns = e0 < p.rot;
  // the lane that holds the other half of this lane's pairs
  const int partner = INTERLEAVED || !turns ? lane : (e0 < half ? lane + half / V : lane - half / V);
  float2 *cs = s_cs[warp];
  float wq[V], wk[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    wq[i] = p.q_weight[e0 + i];
    wk[i] = p.k_weight[e0 + i];
  }
  uint64_t freq[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) freq[i] = lane + 32 * i < half ? turn_fraction(p.inv_freq[lane + 32 * i]) : 0ull;

  const int groups = (H + HPW - 1) / HPW;                 // warp-wide loads per token
  const int per = (groups + p.split - 1) / p.split;       // of which this task takes `per`
  const long long tasks = (long long)p.T * p.split;
  const long long stride = (long long)gridDim.x * kRopeWarps;
  for (long long task = (long long)blockIdx.x * kRopeWarps + warp; task < tasks; task += stride) {
    const long long t = p.split == 1 ? task : task / p.split;
    const int g0 = (int)(task - t * p.split) * per, g1 = min(groups, g0 + per);
    long long position, row = t;
    if (p.positions) {
      position = p.positions[t];
      if (position < 0) continue;  // padding: the row is left alone
      if (p.slots) row = p.slots[t];
    } else {
      const int b = (int)(t / p.tree.N), n = (int)(t - (long long)b * p.tree.N);
      int L = p.prefix_len[b], depth = 0;
      if (L < 0) {
        set_status(p.status, SV_DEV_BAD_PREFIX);
        L = 0;
      }
      if (p.tree.rows) {
        // the sequence's own tree: its parents in the warp's registers, walked by shuffles
        const int32_t *par = p.tree.rows + (size_t)b * p.tree.stride;
        const int p0 = lane < p.tree.N ? par[lane] : -1, p1 = lane + 32 < p.tree.N ? par[lane + 32] : -1;
        int a = n;
        bool ok = __shfl_sync(0xFFFFFFFFu, p0, 0) == -1;
        while (a > 0) {
          const int lo = __shfl_sync(0xFFFFFFFFu, p0, a & 31), hi = __shfl_sync(0xFFFFFFFFu, p1, a & 31);
          const int up = a < 32 ? lo : hi;
          if (up < 0 || up >= a) {
            ok = false;
            break;
          }
          a = up;
          ++depth;
        }
        if (!ok && lane == 0) set_status(p.status, SV_DEV_BAD_TREE);
      } else {
        depth = p.tree.depth[n];
      }
      position = (long long)L + depth;
    }
    const bool write_kv = row >= 0 && row < p.num_rows;
    if (row >= p.num_rows && lane == 0 && g1 == groups) set_status(p.status, SV_DEV_BAD_BLOCK);

    const T *src = static_cast<const T *>(p.qkv) + t * p.ld + e0;
    // the token's cosines and sines, once for all its heads
    if (g0 * HPW < p.Hq + p.Hkv) {
      __syncwarp();
#pragma unroll
      for (int i = 0; i < 2; ++i)
        if (lane + 32 * i < half) cs[lane + 32 * i] = turn_cos_sin(freq[i], position);
      __syncwarp();
    }
    constexpr int NP = INTERLEAVED ? V / 2 : V;  // pairs this lane needs
    float2 rot[NP];
    const int i0 = INTERLEAVED ? e0 / 2 : (e0 < half ? e0 : e0 - half);
#pragma unroll
    for (int i = 0; i < NP; ++i) rot[i] = turns ? cs[i0 + i] : make_float2(1.f, 0.f);

    for (int g = g0; g < g1; g += kRopeUnroll) {
      uint4 raw[kRopeUnroll];
#pragma unroll
      for (int u = 0; u < kRopeUnroll; ++u) {
        const int h = (g + u) * HPW + sub;
        if (g + u < g1 && h < H) raw[u] = __ldcs(reinterpret_cast<const uint4 *>(src + (size_t)h * D));
        else raw[u] = make_uint4(0, 0, 0, 0);
      }
#pragma unroll
      for (int u = 0; u < kRopeUnroll; ++u) {
        if (g + u >= g1) break;  // (the same in the whole warp)
        const int h = (g + u) * HPW + sub;
        float x[V];
        Elem<T>::unpack(raw[u], x);
        float ss = 0.f;
#pragma unroll
        for (int i = 0; i < V; ++i) ss = fmaf(x[i], x[i], ss);
#pragma unroll
        for (int o = LPH / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xFFFFFFFFu, ss, o);
        const float r = rsqrtf(ss * (1.f / D) + p.eps);
        const bool is_q = h < p.Hq;
#pragma unroll
        for (int i = 0; i < V; ++i) x[i] *= r * (is_q ? wq[i] : wk[i]);
        float y[V];
        if constexpr (INTERLEAVED) {
#pragma unroll
          for (int i = 0; i < V / 2; ++i) {
            y[2 * i] = x[2 * i] * rot[i].x - x[2 * i + 1] * rot[i].y;
            y[2 * i + 1] = x[2 * i] * rot[i].y + x[2 * i + 1] * rot[i].x;
          }
        } else {
#pragma unroll
          for (int i = 0; i < V; ++i) {
            const float other = __shfl_sync(0xFFFFFFFFu, x[i], partner);
            y[i] = x[i] * rot[i].x + (e0 < half ? -other : other) * rot[i].y;
          }
        }
        if (h < p.Hq) {
          *reinterpret_cast<uint4 *>(static_cast<T *>(p.q_out) + ((size_t)t * p.Hq + h) * D + e0) = pack_vec<T>(y);
        } else if (h < p.Hq + p.Hkv) {
          if (write_kv)
            *reinterpret_cast<uint4 *>(static_cast<T *>(p.k_out) + ((size_t)row * p.Hkv + (h - p.Hq)) * D + e0) = pack_vec<T>(y);
        } else if (h < H && write_kv) {
          *reinterpret_cast<uint4 *>(static_cast<T *>(p.v_out) + ((size_t)row * p.Hkv + (h - p.Hq - p.Hkv)) * D + e0) = raw[u];
        }
      }
    }
  }
}

template <typename T, int LPH>
cudaError_t launch_rope(const RopeParams &p, int grid, cudaStream_t s) {
  if (p.interleaved) qk_norm_rope_kernel<T, LPH, true><<<grid, kRopeWarps * 32, 0, s>>>(p);
  else qk_norm_rope_kernel<T, LPH, false><<<grid, kRopeWarps * 32, 0, s>>>(p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_qk_norm_rope(sv_dtype dt, int D, RopeParams p, int num_sms, cudaStream_t s) {
  const int lph = D * (dt == SV_BF16 ? 2 : 4) / 16;
  const int groups = (p.Hq + 2 * p.Hkv + 32 / lph - 1) / (32 / lph);
  // few tokens: a token's heads go to several warps, until every SM has a CTA
  const long long want = (long long)num_sms * kRopeWarps;
  long long split = (want + p.T - 1) / p.T;
  p.split = (int)(split < 1 ? 1 : (split > groups ? groups : split));
  const long long ctas = ((long long)p.T * p.split + kRopeWarps - 1) / kRopeWarps;
  const int grid = (int)(ctas < 8ll * num_sms ? ctas : 8ll * num_sms);
  if (dt == SV_BF16) return D == 128 ? launch_rope<bf16, 16>(p, grid, s) : launch_rope<bf16, 8>(p, grid, s);
  return D == 128 ? launch_rope<float, 32>(p, grid, s) : launch_rope<float, 16>(p, grid, s);
}

}  // namespace sv
