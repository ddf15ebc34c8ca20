// Tree attention over a sliding window with sinks in fp32 (sm_103a; FFMA, no tensor cores).
//
// The keys of a node are those of window_attention.cu.  A unit -- a sequence and KV head, up to
// eight of its query rows at a time -- goes to a CTA, or to a cluster of up to eight when there are few
// units; its keys, in chunks of 32 (tree nodes, sinks before the window, window), go round the
// warps, each of which copies its chunk into shared memory of its own and keeps its own running
// maximum, sum and output, so that a short window is one memory round trip and no warp waits for
// another before the merge.  In a chunk lane j scores key j against every row (K rows padded to
// D + 4 floats: conflict-free 16-byte reads, each read once for all rows); for P V lane i holds the
// dimensions i, i + 32, ... and reads the weights of a key as two broadcast vectors.
//
// Bound by latency for few units (5 sequences of 4 heads of 64, 5 rows, window 129: 4.3 us; 7.5 with
// the 5 rows in one CTA).  For many by loads and products that take turns: a warp has room for one
// chunk, so the next one is requested behind the last use of this one, and at D = 128 the chunks of four
// warps leave room for one CTA per SM, so that nothing hides either half (32 KV heads of 20 rows of 128,
// window 2049: 98 us, 6.9 TFLOP/s, about a tenth of the FFMA rate).
#include <atomic>

#include "cluster.cuh"
#include "sv_common.cuh"
#include "sv_internal.h"

namespace sv {

namespace {

constexpr int kF32Keys = 32;   // keys of a chunk: one per lane
constexpr float kF32None = -3e38f;  // a row's maximum before its first key

// The maximum over a warp.
__device__ __forceinline__ float warp_max(float x) {
  float y;
  asm volatile("redux.sync.max.f32 %0, %1, 0xFFFFFFFF;" : "=f"(y) : "f"(x));
  return y;
}

// R floats of shared memory, in as few accesses as they take.
template <int R>
__device__ __forceinline__ void put(float *p, const float (&v)[R]) {
  if constexpr (R == 1) p[0] = v[0];
  else if constexpr (R == 2) *reinterpret_cast<float2 *>(p) = make_float2(v[0], v[1]);
  else
#pragma unroll
    for (int i = 0; i < R; i += 4) *reinterpret_cast<float4 *>(p + i) = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
}
template <int R>
__device__ __forceinline__ void get(const float *p, float (&v)[R]) {
  if constexpr (R == 1) {
    v[0] = p[0];
  } else if constexpr (R == 2) {
    const float2 x = *reinterpret_cast<const float2 *>(p);
    v[0] = x.x;
    v[1] = x.y;
  } else {
#pragma unroll
    for (int i = 0; i < R; i += 4) {
      const float4 x = *reinterpret_cast<const float4 *>(p + i);
      v[i] = x.x;
      v[i + 1] = x.y;
      v[i + 2] = x.z;
      v[i + 3] = x.w;
    }
  }
}

// R: query rows of a CTA (1, 2, 4 or 8); NW: its warps, what one chunk each leaves room for, or two where
// several CTAs share an SM
template <int D>
constexpr int kF32Warps = D == 64 ? 8 : 4;
template <int D, int R, int NW_>
struct F32Layout {
  static constexpr int NW = NW_;
  static constexpr int KS = D + 4;                // row stride of K (floats)
  static constexpr int CHUNK = kF32Keys * (KS + D);  // floats of a warp's chunk
  static constexpr int OFF_P = NW * CHUNK;        // [NW][32][8] weights
  static constexpr int OFF_Q = OFF_P + NW * kF32Keys * R;  // [8][D]
  static constexpr int OFF_M = OFF_Q + R * D;              // [NW][8]
  static constexpr int OFF_L = OFF_M + NW * R;
  static constexpr int OFF_CM = OFF_L + NW * R;            // [8] the CTA's maximum and sum
  static constexpr int OFF_CL = OFF_CM + R;
  static constexpr int SMEM = (OFF_CL + R) * 4;
  static_assert(CHUNK >= R * D, "a warp's outputs merge in the room of its chunk");
};

// The keys: a window's (sv_window_attention), those of the unit's listed pages (sv_sparse_attention), or the sequence's
// whole prefix (sv_shared_attention), which also reports groups that are none.  (Instances of their own: with that
// report for no groups in the window's, 4 requests of 5 nodes, 32:8 heads of 128, window 2049, take 105 us against 98.)
enum F32Kind { kWindowKeys, kListedKeys, kSharedKeys };
template <int D, int R, int NW_, F32Kind KEYS>
__global__ void __launch_bounds__(NW_ * 32) window_f32_kernel(const __grid_constant__ AttnParams p) {
  using Lay = F32Layout<D, R, NW_>;
  constexpr bool LISTED = KEYS == kListedKeys;
  constexpr int NW = Lay::NW, KS = Lay::KS, PL = D / 32;
  extern __shared__ __align__(16) float f32_smem[];
  float *sm = f32_smem;
  float *s_q = sm + Lay::OFF_Q, *s_m = sm + Lay::OFF_M, *s_l = sm + Lay::OFF_L, *s_cm = sm + Lay::OFF_CM,
        *s_cl = sm + Lay::OFF_CL;
  __shared__ int s_par[kMaxNodes], s_lo[R], s_row[R];
  __shared__ uint64_t s_anc[R];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const unsigned C = p.splits, rank = C > 1 ? cluster_rank() : 0;
  const int blocks = (p.M + R - 1) / R, unit = blockIdx.x / C;
  const int mb = unit % blocks, kvh = (unit / blocks) % p.Hkv, bs = unit / blocks / p.Hkv;
  const int b = LISTED ? bs / p.sets : bs, node0 = LISTED ? bs % p.sets * p.set_nodes : 0;
  if (tid < R) {
    const int at = mb * R + tid, node = at / p.G;
    s_row[tid] = at < p.M ? (b * p.N + node0 + node) * p.Hq + kvh * p.G + at - node * p.G : -1;
  }
  __syncthreads();
  wait_previous();
  int L = p.prefix_len[b];
  // rows and tree, on their way before the first chunks
  constexpr int QL = (R * D + NW * 32 - 1) / (NW * 32);
  float qv[QL];
#pragma unroll
  for (int k = 0; k < QL; ++k) {
    const int i = tid + k * NW * 32, row = i < R * D ? s_row[i / D] : -1;
    qv[k] = row >= 0 ? static_cast<const float *>(p.q)[(size_t)row * D + i % D] : 0.f;
  }
  const int parent = tid < p.N ? tree_parent(p.tree, b, tid) : -1;
  if (KEYS == kSharedKeys && tid < 32 && rank == 0 && unit % (blocks * p.Hkv) == 0)
    report_groups(p.group_start, p.shared_len, p.groups, p.B, p.cap, b, L, p.status);
  if (L < 0 || L > p.cap) {
    if (unit % (blocks * p.Hkv) == 0 && node0 == 0 && rank == 0 && tid == 0) set_status(p.status, SV_DEV_BAD_PREFIX);
    L = L < 0 ? 0 : p.cap;
  }
  const int first = LISTED ? 0 : window_first(L, p.window), n_sinks = LISTED ? 0 : min(p.sinks, first);
  // chunks: tree nodes, sinks before the window, window
  const int ct = (p.N + kF32Keys - 1) / kF32Keys, cs = ct + (n_sinks + kF32Keys - 1) / kF32Keys;
  int listed = 0;  // keys of the list
  if constexpr (LISTED) listed = listed_length(p.pages + ((size_t)bs * p.Hkv + kvh) * p.list_len, p.list_len) * p.page_size;
  const int chunks = cs + ((LISTED ? listed : L - first) + kF32Keys - 1) / kF32Keys;
  float *sk = sm + warp * Lay::CHUNK, *sv = sk + kF32Keys * KS, *sp = sm + Lay::OFF_P + warp * kF32Keys * R;
  const float *gkt = static_cast<const float *>(p.k_tree), *gvt = static_cast<const float *>(p.v_tree);
  const float *gkc = static_cast<const float *>(p.cache_k), *gvc = static_cast<const float *>(p.cache_v);

  // chunk c into this warp's room; true in the lanes whose key is there
  auto fetch = [&](int c) -> bool {
    const int base = c < cs ? kF32Keys * (c < ct ? c : c - ct) : first + kF32Keys * (c - cs);
    int key = base + lane;
    const int end = c < ct ? p.N : (c < cs ? n_sinks : L);
    if (LISTED && c >= ct) {  // place `key` of the list: a position, or none
      const int page = key < listed ? p.pages[((size_t)bs * p.Hkv + kvh) * p.list_len + key / p.page_size] : -1;
      const long long at = (long long)page * p.page_size + key % p.page_size;
      key = page >= 0 && at < L ? (int)at : end;
    }
    long long row = -1;
    if (key < end) {
      if (c < ct) {
        row = (long long)b * p.N + key;
      } else if (p.block_table) {
        const int blk = p.block_table[(size_t)b * p.max_blocks + key / p.block_size];
        if (blk >= 0 && blk < p.num_blocks) row = (long long)blk * p.block_size + key % p.block_size;
        else set_status(p.status, SV_DEV_BAD_BLOCK);
      } else {
        row = (long long)b * p.Lmax + key;
      }
    }
    const float *gk = c < ct ? gkt : gkc, *gv = c < ct ? gvt : gvc;
#pragma unroll 8
    for (int f = 0; f < D / 4; ++f) {
      const int i = f * 32 + lane, kk = i / (D / 4), d4 = i % (D / 4);
      const long long r = __shfl_sync(0xFFFFFFFFu, row, kk);
      const size_t off = r < 0 ? 0 : ((size_t)r * p.Hkv + kvh) * D + 4 * d4;
      cp_async_16(sk + kk * KS + 4 * d4, gk + off, r >= 0);  // (zeros where there is no key)
      cp_async_16(sv + kk * D + 4 * d4, gv + off, r >= 0);
    }
    cp_async_commit();
    return row >= 0;
  };
  const int c0 = (int)rank * NW + warp, step = (int)C * NW;
  bool there = false;
  if (c0 < chunks) there = fetch(c0);

  // the rows and what each of them sees, while the first chunks are on their way
  if (tid < kMaxNodes) s_par[tid] = parent;
#pragma unroll
  for (int k = 0; k < QL; ++k)
    if (tid + k * NW * 32 < R * D) s_q[tid + k * NW * 32] = qv[k];
  __syncthreads();
  if (tid < R) {
    const int at = mb * R + tid;
    uint64_t anc = 0;
    int lo = 0, depth;
    if (at < p.M) {
      if (!tree_walk(s_par, node0 + at / p.G, &anc, &depth) && kvh == 0 && rank == 0) set_status(p.status, SV_DEV_BAD_TREE);
      if (!LISTED) {
        lo = window_first(L + depth, p.window);
        anc = window_ancestors(anc, L, p.window, p.sinks);
      }
    }
    s_anc[tid] = anc;
    s_lo[tid] = lo;
  }
  __syncthreads();

  float m[R], l[R], o[R][PL];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    m[r] = kF32None;
    l[r] = 0.f;
#pragma unroll
    for (int i = 0; i < PL; ++i) o[r][i] = 0.f;
  }
  for (int c = c0; c < chunks; c += step) {
    cp_async_wait<0>();
    __syncwarp();
    float s[R];
#pragma unroll
    for (int r = 0; r < R; ++r) s[r] = 0.f;
    const float4 *kr = reinterpret_cast<const float4 *>(sk + lane * KS), *qr = reinterpret_cast<const float4 *>(s_q);
#pragma unroll 4
    for (int d4 = 0; d4 < D / 4; ++d4) {
      const float4 k4 = kr[d4];
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const float4 q4 = qr[r * (D / 4) + d4];
        s[r] = fmaf(q4.x, k4.x, s[r]);
        s[r] = fmaf(q4.y, k4.y, s[r]);
        s[r] = fmaf(q4.z, k4.z, s[r]);
        s[r] = fmaf(q4.w, k4.w, s[r]);
      }
    }
    const int key = (c < cs ? kF32Keys * (c < ct ? c : c - ct) : first + kF32Keys * (c - cs)) + lane;
    float w[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const bool see = there && (c < ct ? ((s_anc[r] >> (key & 63)) & 1ull) != 0
                                        : (LISTED || c < cs || key >= s_lo[r] || key < p.sinks));
      const float x = see ? s[r] * p.scale_log2 : -INFINITY;
      const float top = fmaxf(warp_max(x), m[r]);
      const float a = exp2f(m[r] - top);
      m[r] = top;
      w[r] = see ? exp2f(x - top) : 0.f;
      l[r] = l[r] * a + w[r];  // (each lane its own keys; summed over the lanes at the end)
#pragma unroll
      for (int i = 0; i < PL; ++i) o[r][i] *= a;
    }
    put<R>(sp + lane * R, w);
    __syncwarp();
#pragma unroll 4
    for (int j = 0; j < kF32Keys; ++j) {
      float wj[R];
      get<R>(sp + j * R, wj);
#pragma unroll
      for (int i = 0; i < PL; ++i) {
        const float v = sv[j * D + lane + 32 * i];
#pragma unroll
        for (int r = 0; r < R; ++r) o[r][i] = fmaf(wj[r], v, o[r][i]);
      }
    }
    __syncwarp();  // every lane is done with the chunk
    if (c + step < chunks) there = fetch(c + step);
  }

  // merge the warps: outputs against the CTA's maximum, in the room of the chunks
#pragma unroll
  for (int r = 0; r < R; ++r) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) l[r] += __shfl_xor_sync(0xFFFFFFFFu, l[r], off);
    if (lane == 0) {
      s_m[warp * R + r] = m[r];
      s_l[warp * R + r] = l[r];
    }
  }
  __syncthreads();
#pragma unroll
  for (int r = 0; r < R; ++r) {
    float top = kF32None;
#pragma unroll
    for (int k = 0; k < NW; ++k) top = fmaxf(top, s_m[k * R + r]);
    const float a = exp2f(m[r] - top);
#pragma unroll
    for (int i = 0; i < PL; ++i) sk[r * D + lane + 32 * i] = o[r][i] * a;
  }
  if (tid < R) {
    float top = kF32None, sum = 0.f;
#pragma unroll
    for (int k = 0; k < NW; ++k) top = fmaxf(top, s_m[k * R + tid]);
#pragma unroll
    for (int k = 0; k < NW; ++k) sum += exp2f(s_m[k * R + tid] - top) * s_l[k * R + tid];
    s_cm[tid] = top;
    s_cl[tid] = sum;
  }
  __syncthreads();
  auto store = [&](int r, int d4, float4 x) {
    const int row = s_row[r];
    if (row >= 0) *reinterpret_cast<float4 *>(static_cast<float *>(p.out) + (size_t)row * D + 4 * d4) = x;
  };
  for (int u = tid; u < R * (D / 4); u += NW * 32) {
    const int r = u / (D / 4), d4 = u % (D / 4);
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int k = 0; k < NW; ++k) {
      const float4 y = *reinterpret_cast<const float4 *>(sm + k * Lay::CHUNK + r * D + 4 * d4);
      x.x += y.x;
      x.y += y.y;
      x.z += y.z;
      x.w += y.w;
    }
    if (C > 1) {
      *reinterpret_cast<float4 *>(sm + r * D + 4 * d4) = x;
    } else {
      const float inv = s_cl[r] > 0.f ? 1.f / s_cl[r] : 0.f;
      store(r, d4, make_float4(x.x * inv, x.y * inv, x.z * inv, x.w * inv));
    }
  }
  if (C > 1) cluster_merge<D>(sm, D, s_cm, s_cl, R, C, rank, kF32None, sm + Lay::CHUNK, store);
}

template <int D, int R, int NW, F32Kind KEYS>
cudaError_t launch_f32_d(const AttnParams &p, long long ctas, cudaStream_t s) {
  using Lay = F32Layout<D, R, NW>;
  static_assert(Lay::SMEM <= 227 * 1024, "shared memory");
  static std::atomic<bool> attr[64];
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev < 0 || dev >= 64 || !attr[dev].load()) {
    const cudaError_t e =
        cudaFuncSetAttribute(window_f32_kernel<D, R, NW, KEYS>, cudaFuncAttributeMaxDynamicSharedMemorySize, Lay::SMEM);
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < 64) attr[dev].store(true);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)ctas);
  cfg.blockDim = dim3(Lay::NW * 32);
  cfg.dynamicSmemBytes = Lay::SMEM;
  cfg.stream = s;
  cudaLaunchAttribute at[2];
  at[0] = close_launch();
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = (unsigned)p.splits;
  at[1].val.clusterDim.y = 1;
  at[1].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = p.splits > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, window_f32_kernel<D, R, NW, KEYS>, p);
}

// `kv_units` sequences (or sets of nodes) and KV heads of p.M rows, against up to `keys` keys.
template <F32Kind KEYS>
cudaError_t launch_f32(AttnParams p, long long kv_units, long long keys, int num_sms, cudaStream_t s) {
  // Rows of a CTA and CTAs per unit (splits): few rows are done sooner, many read K and V fewer
  // times.  As fitted to measurements (us, 4 to 128 KV heads of 1 to 64 rows, windows 17 to 2049; one
  // CTA per SM): a wave of CTAs takes 3.4 + 0.45 rows and 2.3 + 0.25 rows for every further chunk of
  // its warps, a cluster 2 more.  20 KV heads of 5 rows of 64, window 129: 4.7 us with a row each
  // against 7.8 with eight; 32 of 20 rows of 128, window 2049, 98 with eight (two take 128).
  // Many short lists (26 nodes of 8 heads of 128 with a page of 16 each, 8 sequences: 1664 units of two
  // chunks, 20.6 us against 49.7) have two warps to a CTA, of which three (heads of 64: six) share an SM.
  const int full = p.D == 64 ? 8 : 4;
  const int chunks = (int)(keys / kF32Keys) + (p.N + p.sinks) / kF32Keys + 2;
  int rows = 1, warps = full;
  long long units = 0;
  double best = 0;
  for (int w = full; w >= (KEYS == kListedKeys ? 2 : full); w = w > 2 ? 2 : 0)
    for (int r = 1; r <= 8 && (r == 1 || r < 2 * p.M); r *= 2)
      for (int c = 1; c <= (w == full ? 8 : 1); c *= 2) {
        const long long u = kv_units * ((p.M + r - 1) / r);
        if (c == 8 && u * c > num_sms * 2 / 3) break;  // 16 clusters of 8 do not find room together
        const long long places = (long long)num_sms * (w == full ? 1 : p.D == 64 ? 6 : 3);
        const double waves = (double)((u * c + places - 1) / places);
        const int further = (chunks + c * w - 1) / (c * w) - 1;
        const double cost = waves * (3.4 + 0.45 * r + further * (2.3 + 0.25 * r) + (c > 1 ? 2 : 0));
        if (units == 0 || cost < best) {
          best = cost;
          rows = r;
          units = u;
          warps = w;
          p.splits = c;
        }
      }
  const long long ctas = units * p.splits;
  if (ctas > INT32_MAX) return cudaErrorInvalidValue;
  if constexpr (KEYS == kListedKeys) {
    if (warps == 2) {
      switch (rows * 1000 + p.D) {
        case 1064: return launch_f32_d<64, 1, 2, kListedKeys>(p, ctas, s);
        case 2064: return launch_f32_d<64, 2, 2, kListedKeys>(p, ctas, s);
        case 4064: return launch_f32_d<64, 4, 2, kListedKeys>(p, ctas, s);
        case 8064: return launch_f32_d<64, 8, 2, kListedKeys>(p, ctas, s);
        case 1128: return launch_f32_d<128, 1, 2, kListedKeys>(p, ctas, s);
        case 2128: return launch_f32_d<128, 2, 2, kListedKeys>(p, ctas, s);
        case 4128: return launch_f32_d<128, 4, 2, kListedKeys>(p, ctas, s);
        default: return launch_f32_d<128, 8, 2, kListedKeys>(p, ctas, s);
      }
    }
  }
  switch (rows * 1000 + p.D) {
    case 1064: return launch_f32_d<64, 1, kF32Warps<64>, KEYS>(p, ctas, s);
    case 2064: return launch_f32_d<64, 2, kF32Warps<64>, KEYS>(p, ctas, s);
    case 4064: return launch_f32_d<64, 4, kF32Warps<64>, KEYS>(p, ctas, s);
    case 8064: return launch_f32_d<64, 8, kF32Warps<64>, KEYS>(p, ctas, s);
    case 1128: return launch_f32_d<128, 1, kF32Warps<128>, KEYS>(p, ctas, s);
    case 2128: return launch_f32_d<128, 2, kF32Warps<128>, KEYS>(p, ctas, s);
    case 4128: return launch_f32_d<128, 4, kF32Warps<128>, KEYS>(p, ctas, s);
    default: return launch_f32_d<128, 8, kF32Warps<128>, KEYS>(p, ctas, s);
  }
}

}  // namespace

cudaError_t launch_window_attention_f32(AttnParams p, int num_sms, cudaStream_t s) {
  const int span = p.window - 1 < p.cap ? p.window - 1 : p.cap;
  return launch_f32<kWindowKeys>(p, (long long)p.B * p.Hkv, span, num_sms, s);
}

cudaError_t launch_shared_attention_f32(AttnParams p, const ListArgs &l, int num_sms, cudaStream_t s) {
  p.group_start = l.group_start;
  p.shared_len = l.shared_len;
  p.groups = l.groups;
  return launch_f32<kSharedKeys>(p, (long long)p.B * p.Hkv, p.cap, num_sms, s);
}

cudaError_t launch_sparse_attention_f32(AttnParams p, const ListArgs &l, int num_sms, cudaStream_t s) {
  p.pages = l.pages;
  p.list_len = l.list_len;
  p.page_size = l.page_size;
  p.sets = l.sets;
  p.set_nodes = p.N / l.sets;
  p.M = p.set_nodes * p.G;
  return launch_f32<kListedKeys>(p, (long long)p.B * l.sets * p.Hkv, (long long)l.list_len * l.page_size, num_sms, s);
}

}  // namespace sv
