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
// position wraps exactly: no argument reduction and no loss at far positions (off by less than
// 2^-64 of a turn per position).  The nearest quarter turn comes off in
// integers, so that the sine and cosine are taken of at most an eighth of a turn.
//
// A warp takes a token (or, when there are few tokens, a part of its heads) and reads whole
// heads with 16-byte loads, the next four in flight while four are worked on, across tokens
// too.  Sines and cosines are computed once per token; with the weights they make two factors
// per element, so that a head costs
//   out_i = r (x_i A_i + x_j B_i),  j the other element of i's pair, r = 1 / sqrt(mean + eps),
// and the other lane's x_j comes as the raw 16 bits it was loaded as.  It is bound by HBM:
// each element is read once and written once.  32768 tokens of 32:8 heads of 128 in bf16 take
// 127 us, 6.32 TB/s, 93 % of the measured copy rate; 171 us before the loads ran ahead of the
// work and the factors were made per token; 135 us with 16 instead of 20 warps per SM; 140 us
// with stores that stay in L2 (the outputs of a prompt exceed it).
#include "sv_common.cuh"
#include "sv_internal.h"

namespace sv {

namespace {

constexpr int kRopeWarps = 4;
constexpr int kRopeCtas = 5;   // resident per SM
constexpr int kRopeBatch = 4;  // warp-wide loads worked on together (as many are in flight)

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

// The fraction of a turn per position, of 2^64: f / (2 pi) mod 1 with f = m 2^e, m a 53-bit integer, as
// the 117-bit product of m and 2^66 / (2 pi), shifted by e - 2 places (off by less than 2^-64 and
// 2^-64 f).  In integers, once per CTA: products and roundings in double take 16 cycles of the SM per
// warp each.  With that, and the first token requested before the weights: 384 tokens 5.8 -> 5.1 us,
// 4096 21.7 -> 21.0, 32768 129 -> 127.4.
__device__ __forceinline__ uint64_t turn_fraction(double f) {
  constexpr uint64_t kPerTurn = 0xA2F9836E4E44152Aull;  // 2^66 / (2 pi)
  const uint64_t bits = (uint64_t)__double_as_longlong(f);
  const int field = (int)(bits >> 52) & 2047, shift = 1077 - (field ? field : 1);
  const uint64_t m = (bits & 0xFFFFFFFFFFFFFull) | (field ? 1ull << 52 : 0ull);
  const uint64_t lo = m * kPerTurn, hi = __umul64hi(m, kPerTurn);
  uint64_t x;
  if (shift <= 0) x = shift > -64 ? lo << -shift : 0ull;
  else if (shift < 64) x = lo >> shift | hi << (64 - shift);
  else x = shift < 128 ? hi >> (shift - 64) : 0ull;
  return bits >> 63 ? 0ull - x : x;
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

// The position of token t and, in the tree form, of the node that it is.
__device__ __forceinline__ long long token_position(const RopeParams &p, long long t) {
  if (p.positions) return p.positions[t];
  const int lane = threadIdx.x & 31;
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
  return (long long)L + depth;
}

// LPH lanes hold one head of D = LPH * 16 / sizeof(T) elements, 16 bytes each.
template <typename T, int LPH, bool INTERLEAVED>
__global__ void __launch_bounds__(kRopeWarps * 32, kRopeCtas) qk_norm_rope_kernel(const __grid_constant__ RopeParams p) {
  constexpr int V = Elem<T>::kVec;
  constexpr int D = LPH * V, HPW = 32 / LPH;  // heads per warp-wide load
  constexpr int U = kRopeBatch;
  __shared__ __align__(16) float2 s_cs[kRopeWarps][64];
  __shared__ __align__(16) float s_w[2][128];
  __shared__ uint64_t s_turn[64];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int l = lane % LPH, sub = lane / LPH, e0 = l * V;
  const int half = p.rot >> 1;
  const bool turns = e0 < p.rot, second = !INTERLEAVED && e0 >= half;
  // the lane that holds the other elements of this lane's pairs
  const int partner = INTERLEAVED || !turns ? lane : (second ? lane - half / V : lane + half / V);
  const int j0 = (partner % LPH) * V;
  float2 *cs = s_cs[warp];
  wait_previous();
  // (requested before the first token, used behind its loads)
  const bool holds = threadIdx.x < D;
  const float qw = holds ? p.q_weight[threadIdx.x] : 0.f, kw = holds ? p.k_weight[threadIdx.x] : 0.f;
  const double turn = threadIdx.x < 64 && (int)threadIdx.x < half ? p.inv_freq[threadIdx.x] : 0.0;

  // a token's batches: query heads, key heads, value heads (none mixes two kinds)
  const int nq = (p.Hq + HPW * U - 1) / (HPW * U), nk = (p.Hkv + HPW * U - 1) / (HPW * U), nb = nq + 2 * nk;
  const int per = (nb + p.split - 1) / p.split;  // of which a task takes `per`
  const long long tasks = (long long)p.T * p.split, stride = (long long)gridDim.x * kRopeWarps;
  long long task = (long long)blockIdx.x * kRopeWarps + warp;
  auto token_of = [&](long long k) { return p.split == 1 ? k : k / p.split; };
  auto first_batch = [&](long long k) { return p.split == 1 ? 0 : (int)(k - token_of(k) * p.split) * per; };
  auto last_batch = [&](int b0) { return min(nb, b0 + per); };

  auto load = [&](uint4 (&raw)[U], long long t, int bi) {
    const int kind = bi < nq ? 0 : (bi < nq + nk ? 1 : 2), heads = kind == 0 ? p.Hq : p.Hkv;
    const int h0 = (bi - (kind == 0 ? 0 : (kind == 1 ? nq : nq + nk))) * HPW * U + sub;
    const T *src = static_cast<const T *>(p.qkv) + t * p.ld + e0 +
                   (size_t)(h0 + (kind == 0 ? 0 : (kind == 1 ? p.Hq : p.Hq + p.Hkv))) * D;
#pragma unroll
    for (int u = 0; u < U; ++u)
      raw[u] = h0 + u * HPW < heads ? load_streamed(reinterpret_cast<const uint4 *>(src + u * HPW * D)) : make_uint4(0, 0, 0, 0);
  };

  // the task at hand (a token, or a part of its batches), its place in the cache, its position
  long long t = 0, row = 0, position = 0;
  int bi = 0, b1 = 0;
  bool write_kv = false;
  uint4 raw[2][U];
  auto begin = [&]() -> bool {  // the next task that is not padding; false at the end
    for (; task < tasks; task += stride) {
      bi = first_batch(task);
      b1 = last_batch(bi);
      if (bi >= b1) continue;
      t = token_of(task);
      position = token_position(p, t);
      if (p.positions && position < 0) continue;  // padding: the row is left alone
      row = p.slots ? (long long)p.slots[t] : t;
      write_kv = row >= 0 && row < p.num_rows;
      if (row >= p.num_rows && lane == 0 && b1 == nb) set_status(p.status, SV_DEV_BAD_BLOCK);
      task += stride;
      return true;
    }
    return false;
  };
  auto angles = [&]() {  // the task's cosines and sines, once for all its heads
    if (bi >= nq + nk) return;
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 2; ++i)
      if (lane + 32 * i < half) cs[lane + 32 * i] = turn_cos_sin(s_turn[lane + 32 * i], position);
    __syncwarp();
  };
  const bool any = begin();
  if (any) load(raw[0], t, bi);
  if (holds) {
    s_w[0][threadIdx.x] = qw;
    s_w[1][threadIdx.x] = kw;
  }
  if (threadIdx.x < 64) s_turn[threadIdx.x] = turn_fraction(turn);
  __syncthreads();
  if (!any) return;
  angles();
  int kind = -1;
  float2 A[V / 2], B[V / 2];

  // one batch: work on raw[K] while raw[K ^ 1] is loaded.  False after the last one.
  auto batch = [&](uint4 (&now)[U], uint4 (&next)[U]) -> bool {
    const long long ct = t, crow = row;
    const int cb = bi;
    const bool ckv = write_kv;
    // the next batch, of this task or the next one
    bool more = true, fresh = false;
    if (++bi == b1) {
      more = begin();
      fresh = true;
    }
    if (more) load(next, t, bi);

    const int ck = cb < nq ? 0 : (cb < nq + nk ? 1 : 2), heads = ck == 0 ? p.Hq : p.Hkv;
    const int h0 = (cb - (ck == 0 ? 0 : (ck == 1 ? nq : nq + nk))) * HPW * U + sub;
    if (ck != kind && ck < 2) {
      // the factors of this lane's elements for this kind of head and this token
      const int i0 = INTERLEAVED ? e0 / 2 : (second ? e0 - half : e0);
      float a[V], b[V];
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const float2 c = turns ? cs[i0 + (INTERLEAVED ? i / 2 : i)] : make_float2(1.f, 0.f);
        const int j = INTERLEAVED ? e0 + (i ^ 1) : j0 + i;
        a[i] = s_w[ck][e0 + i] * c.x;
        b[i] = s_w[ck][j] * ((INTERLEAVED ? (i & 1) != 0 : second) ? c.y : -c.y);
      }
#pragma unroll
      for (int i = 0; i < V / 2; ++i) {
        A[i] = make_float2(a[2 * i], a[2 * i + 1]);
        B[i] = make_float2(b[2 * i], b[2 * i + 1]);
      }
    }
    kind = ck;
    T *dst = ck == 0 ? static_cast<T *>(p.q_out) + ((size_t)ct * p.Hq + h0) * D + e0
                     : static_cast<T *>(ck == 1 ? p.k_out : p.v_out) + ((size_t)(ckv ? crow : 0) * p.Hkv + h0) * D + e0;
    const bool writes = ck == 0 || ckv;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      uint4 out = now[u];
      if (ck < 2) {
        float x[V], xj[V];
        Elem<T>::unpack(now[u], x);
        if constexpr (INTERLEAVED) {
#pragma unroll
          for (int i = 0; i < V; ++i) xj[i] = x[i ^ 1];
        } else {
          const uint4 o = make_uint4(__shfl_sync(0xFFFFFFFFu, now[u].x, partner), __shfl_sync(0xFFFFFFFFu, now[u].y, partner),
                                     __shfl_sync(0xFFFFFFFFu, now[u].z, partner), __shfl_sync(0xFFFFFFFFu, now[u].w, partner));
          Elem<T>::unpack(o, xj);
        }
        float2 s2 = make_float2(0.f, 0.f);
#pragma unroll
        for (int i = 0; i < V / 2; ++i) s2 = __ffma2_rn(make_float2(x[2 * i], x[2 * i + 1]), make_float2(x[2 * i], x[2 * i + 1]), s2);
        float ss = s2.x + s2.y;
#pragma unroll
        for (int o = LPH / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xFFFFFFFFu, ss, o);
        const float r = rsqrtf(fmaf(ss, 1.f / D, p.eps));
        float y[V];
#pragma unroll
        for (int i = 0; i < V / 2; ++i) {
          const float2 z = mul2(__ffma2_rn(make_float2(xj[2 * i], xj[2 * i + 1]), B[i],
                                           mul2(make_float2(x[2 * i], x[2 * i + 1]), A[i])),
                                make_float2(r, r));
          y[2 * i] = z.x;
          y[2 * i + 1] = z.y;
        }
        out = pack_vec<T>(y);
      }
      if (writes && h0 + u * HPW < heads) __stcs(reinterpret_cast<uint4 *>(dst + u * HPW * D), out);
    }
    if (fresh && more) {
      angles();
      kind = -1;
    }
    return more;
  };
  while (batch(raw[0], raw[1]) && batch(raw[1], raw[0])) {
  }
}

template <typename T, int LPH>
cudaError_t launch_rope(const RopeParams &p, int grid, cudaStream_t s) {
  return launch_close(p.interleaved ? qk_norm_rope_kernel<T, LPH, true> : qk_norm_rope_kernel<T, LPH, false>, dim3(grid),
                      kRopeWarps * 32, 0, s, p);
}

}  // namespace

cudaError_t launch_qk_norm_rope(sv_dtype dt, int D, RopeParams p, int num_sms, cudaStream_t s) {
  const int lph = D * (dt == SV_BF16 ? 2 : 4) / 16;
  const int heads = 32 / lph * kRopeBatch;  // of a batch
  const int batches = (p.Hq + heads - 1) / heads + 2 * ((p.Hkv + heads - 1) / heads);
  // few tokens: a token's batches of heads go to several warps, until every SM has eight (384
  // tokens of 32:8 heads 6.0 us, with four 6.6, with 16 5.7; 777 fp32 tokens 5.1, 5.7, 6.3)
  const long long want = 8ll * num_sms;
  long long split = (want + p.T - 1) / p.T;
  p.split = (int)(split < 1 ? 1 : (split > batches ? batches : split));
  const long long ctas = ((long long)p.T * p.split + kRopeWarps - 1) / kRopeWarps;
  const long long resident = (long long)kRopeCtas * num_sms;
  const int grid = (int)(ctas < resident ? ctas : resident);
  if (dt == SV_BF16) return D == 128 ? launch_rope<bf16, 16>(p, grid, s) : launch_rope<bf16, 8>(p, grid, s);
  return D == 128 ? launch_rope<float, 32>(p, grid, s) : launch_rope<float, 16>(p, grid, s);
}

}  // namespace sv
