// Pages that a query looks at (sm_103a): bounds of the pages' keys, scores of the pages against queries, and
// the selection of the best ones, for sv_sparse_attention.
//
// Bounds: for a page (16 or more keys of a KV head) the least and the largest value of each of its D
// channels.  Of any key k of the page, q . k <= sum_d max(q_d lo_d, q_d hi_d) =
//   sum_d max(q_d, 0) hi_d + min(q_d, 0) lo_d,
// so that a page whose score is low holds no key that matters to q, and the score is two products of
// matrices.  Read once, K is what bounds the first; the bounds (1/8 of K and less) the second.
#include <algorithm>
#include <atomic>
#include <cfloat>
#include <climits>

#include "sv_common.cuh"
#include "sv_internal.h"

namespace sv {

namespace {

// ---------------------------------------------------------------------- bounds

constexpr int kBoundThreads = 128;
constexpr int kBoundRows = 16;  // rows on their way at a time

// Two elements' least and largest; a NaN is kept.
__device__ __forceinline__ uint32_t min_bf16x2_nan(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("min.NaN.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
__device__ __forceinline__ uint32_t max_bf16x2_nan(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
__device__ __forceinline__ float min_nan(float a, float b) {
  float d;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}
__device__ __forceinline__ float max_nan(float a, float b) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}
template <bool F32>
__device__ __forceinline__ uint32_t low_of(uint32_t a, uint32_t b) {
  if constexpr (F32) return __float_as_uint(min_nan(__uint_as_float(a), __uint_as_float(b)));
  else return min_bf16x2_nan(a, b);
}
template <bool F32>
__device__ __forceinline__ uint32_t high_of(uint32_t a, uint32_t b) {
  if constexpr (F32) return __float_as_uint(max_nan(__uint_as_float(a), __uint_as_float(b)));
  else return max_bf16x2_nan(a, b);
}

// A thread per 16 bytes of a page's rows: consecutive threads read consecutive pieces of a row.  A step is 16
// rows of a page, which go through shared memory of the thread's own (cp.async), the next step's on their
// way while one is worked on: 192 KB per SM, where registers hold less than half of that.
template <bool F32>
__global__ void __launch_bounds__(kBoundThreads) page_bounds_kernel(const __grid_constant__ BoundParams p) {
  extern __shared__ __align__(16) uint4 bound_smem[];  // [2][kBoundRows][kBoundThreads]
  wait_previous();
  const int b = blockIdx.y;
  int L = p.prefix_len[b];
  if (L < 0 || L > p.cap) {
    if (blockIdx.x == 0 && threadIdx.x == 0) set_status(p.status, SV_DEV_BAD_PREFIX);
    L = L < 0 ? 0 : p.cap;
  }
  const int start = p.start ? max(p.start[b], 0) : 0;
  if (start >= L) return;
  const int first = start / p.page_size, pages = (L + p.page_size - 1) / p.page_size - first;
  const long long items = (long long)pages * p.vecs, stride = (long long)gridDim.x * kBoundThreads;
  // an item: a page and a piece of its rows
  struct Item {
    const uint4 *src;
    uint4 *dst;
    int rows;
  };
  long long next = (long long)blockIdx.x * kBoundThreads + threadIdx.x;
  auto take = [&]() -> Item {
    for (; next < items; next += stride) {
      const int page = first + (int)(next / p.vecs), v = (int)(next % p.vecs);
      long long row = (long long)b * p.Lmax + (long long)page * p.page_size, out = (long long)b * p.seq_pages + page;
      if (p.block_table) {
        const int blk = p.block_table[(size_t)b * p.max_blocks + page];
        if (blk < 0 || blk >= p.num_blocks) {
          if (v == 0) set_status(p.status, SV_DEV_BAD_BLOCK);
          continue;
        }
        row = (long long)blk * p.page_size;
        out = blk;
      }
      next += stride;
      // head h: D least values, then D largest
      const int h = v / p.head_vecs, d = v % p.head_vecs;
      return {static_cast<const uint4 *>(p.k) + (size_t)row * p.vecs + v,
              static_cast<uint4 *>(p.bounds) + ((size_t)out * p.vecs + (size_t)h * p.head_vecs) * 2 + d, min(p.page_size, L - page * p.page_size)};
    }
    return {nullptr, nullptr, 0};
  };
  uint4 *mine = bound_smem + threadIdx.x;
  auto ask = [&](const Item &it, int r0, int buf) {
#pragma unroll
    for (int r = 0; r < kBoundRows; ++r)
      if (r0 + r < it.rows) cp_async_16(mine + (buf * kBoundRows + r) * kBoundThreads, it.src + (size_t)(r0 + r) * p.vecs, true);
    cp_async_commit();
  };
  Item cur = take(), ahead{};
  int r0 = 0, buf = 0;
  if (cur.rows > 0) ask(cur, 0, 0);
  uint4 lo, hi;
  while (cur.rows > 0) {
    const bool last = r0 + kBoundRows >= cur.rows;
    if (last) ahead = take();
    if (last ? ahead.rows > 0 : true) ask(last ? ahead : cur, last ? 0 : r0 + kBoundRows, buf ^ 1);
    else cp_async_commit();
    cp_async_wait<1>();
    const uint4 *x = mine + buf * kBoundRows * kBoundThreads;
    if (r0 == 0) lo = hi = x[0];
#pragma unroll
    for (int r = 0; r < kBoundRows; ++r)
      if (r0 + r < cur.rows) {
        const uint4 y = x[r * kBoundThreads];
        lo = make_uint4(low_of<F32>(lo.x, y.x), low_of<F32>(lo.y, y.y), low_of<F32>(lo.z, y.z), low_of<F32>(lo.w, y.w));
        hi = make_uint4(high_of<F32>(hi.x, y.x), high_of<F32>(hi.y, y.y), high_of<F32>(hi.z, y.z), high_of<F32>(hi.w, y.w));
      }
    if (last) {
      cur.dst[0] = lo;
      cur.dst[p.head_vecs] = hi;
      cur = ahead;
      r0 = 0;
    } else {
      r0 += kBoundRows;
    }
    buf ^= 1;
  }
  cp_async_wait<0>();
}

// -------------------------------------------------- scores (bf16: page_scores_tc.cu)

// fp32: a warp per page, lanes over the channels.
template <int D>
__global__ void __launch_bounds__(256) page_scores_f32_kernel(const __grid_constant__ ScoreParams p) {
  constexpr int PL = D / 32;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int bh = blockIdx.x / p.splits, part = blockIdx.x % p.splits, h = bh % p.Hkv, b = bh / p.Hkv;
  wait_previous();
  int L = p.prefix_len[b];
  const int most = (int)min((long long)INT_MAX, (long long)p.P * p.page_size);
  if (L < 0 || L > most) {
    if (h == 0 && part == 0 && threadIdx.x == 0) set_status(p.status, SV_DEV_BAD_PREFIX);
    L = L < 0 ? 0 : most;
  }
  const int pages = (int)(((long long)L + p.page_size - 1) / p.page_size);
  float *out = p.out + (size_t)b * p.sets * p.Hkv * p.P + (size_t)h * p.P;
  for (int page = part * 8 + warp; page < p.P; page += p.splits * 8) {
    long long row = -1;
    if (page < pages) {
      if (!p.block_table) {
        row = (long long)b * p.P + page;
      } else {
        const int blk = p.block_table[(size_t)b * p.P + page];
        if (blk >= 0 && blk < p.num_blocks) row = blk;
        else if (h == 0 && lane == 0) set_status(p.status, SV_DEV_BAD_BLOCK);
      }
    }
    float lo[PL], hi[PL];
    const float *src = static_cast<const float *>(p.bounds) + ((size_t)max(row, 0ll) * p.Hkv + h) * 2 * D + lane;
#pragma unroll
    for (int i = 0; i < PL; ++i) {
      lo[i] = row >= 0 ? src[32 * i] : 0.f;
      hi[i] = row >= 0 ? src[D + 32 * i] : 0.f;
    }
    for (int set = 0; set < p.sets; ++set) {
      float best = -INFINITY;
      for (int r = 0; r < p.set_nodes * p.G && row >= 0; ++r) {
        const float *q = static_cast<const float *>(p.q) + (((size_t)b * p.N + set * p.set_nodes + r / p.G) * p.Hq + h * p.G + r % p.G) * D + lane;
        float x = 0.f;
#pragma unroll
        for (int i = 0; i < PL; ++i) {
          const float y = q[32 * i];
          x = fmaf(max_nan(y, 0.f), hi[i], x);
          x = fmaf(min_nan(y, 0.f), lo[i], x);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xFFFFFFFFu, x, o);
        best = max_nan(best, x);
      }
      if (lane == 0) out[(size_t)set * p.Hkv * p.P + page] = best;
    }
  }
}

// ------------------------------------------------------------------- selection

// Order-preserving key of a score: larger for larger scores, the largest for a NaN; the two zeros are one.
__device__ __forceinline__ uint32_t score_key(float x) {
  if (x != x) return 0xFFFFFFFFu;
  const uint32_t u = __float_as_uint(x + 0.f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// A CTA per list.  One histogram of 256 equal parts of the scores' range gives the part in which the last
// place falls.  What is above it is chosen; what is in it are candidates, few as a rule, of which each counts
// those before it (or, many of them, digits of 8 bits of their keys decide, and of those equal to the end
// the lower pages).  (The highest bits in which the keys differ as the first digit: scores of both signs then
// meet in a few of its words, and 2560 lists of up to 2048 scores take 23 us for the atomics instead of 18.3;
// without atomics, by counts against seven pivots at a time until few scores are left, 25.3.)
// The chosen pages are bits of words, from which a lane puts out those of its word.
constexpr int kSelectThreads = 512;  // at most
constexpr int kCandidates = 512;     // of a list; more of them are looked up among all scores again

struct SelectWords {
  uint32_t over, tie;  // chosen; equal to the threshold
};

__global__ void __launch_bounds__(kSelectThreads) select_pages_kernel(const __grid_constant__ SelectParams p) {
  extern __shared__ __align__(8) uint32_t sel_smem[];
  SelectWords *words = reinterpret_cast<SelectWords *>(sel_smem);                    // [ceil(P / 32)]
  float *score = reinterpret_cast<float *>(sel_smem) + 2 * ((p.P + 31) / 32);        // [P]
  __shared__ uint16_t cand[kCandidates];
  __shared__ uint32_t hist[2][256], s_bin, s_left, s_whole, s_cand;
  __shared__ float red[2][32];
  __shared__ int above[32], equal[32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, T = blockDim.x, warps = T >> 5;
  const long long list = blockIdx.x;
  const int b = (int)(list / p.lists);
  for (int i = tid; i < 256; i += T) hist[0][i] = 0;
  if (tid == 0) s_cand = 0;
  wait_previous();
  int L = p.prefix_len[b];
  const int most = (int)min((long long)INT_MAX, (long long)p.P * p.page_size);
  if (L < 0 || L > most) {
    if (list % p.lists == 0 && tid == 0) set_status(p.status, SV_DEV_BAD_PREFIX);
    L = L < 0 ? 0 : most;
  }
  const int pages = (int)(((long long)L + p.page_size - 1) / p.page_size);
  int32_t *out = p.out + list * p.K;
  if (pages <= p.K) {
    for (int i = tid; i < p.K; i += T) out[i] = i < pages ? i : -1;
    return;
  }
  // pages [m0, m1) compete for `left` places
  const int m0 = p.first, m1 = pages - p.last;
  int left = p.K - p.first - p.last;
  const float *x = p.scores + list * p.P;
  float least = FLT_MAX, largest = -FLT_MAX;  // of the finite ones
#pragma unroll 8
  for (int i = m0 + tid; i < m1; i += T) {
    const float v = x[i];
    score[i] = v;
    if (fabsf(v) <= FLT_MAX) {
      least = fminf(least, v);
      largest = fmaxf(largest, v);
    }
  }
  asm volatile("redux.sync.min.f32 %0, %0, 0xFFFFFFFF;" : "+f"(least));
  asm volatile("redux.sync.max.f32 %0, %0, 0xFFFFFFFF;" : "+f"(largest));
  if (lane == 0) red[0][warp] = least, red[1][warp] = largest;
  __syncthreads();
  least = lane < warps ? red[0][lane] : FLT_MAX;
  largest = lane < warps ? red[1][lane] : -FLT_MAX;
  asm volatile("redux.sync.min.f32 %0, %0, 0xFFFFFFFF;" : "+f"(least));
  asm volatile("redux.sync.max.f32 %0, %0, 0xFFFFFFFF;" : "+f"(largest));
  // the part of the range, growing with the score; infinities and NaN are at the ends
  const float range = largest - least, scale = range > 0.f && range <= FLT_MAX ? 255.f / range : 0.f;
  auto bin_of = [&](float v) -> int {
    if (!(fabsf(v) <= FLT_MAX)) return v == -INFINITY ? 0 : 255;
    return min(255, (int)((v - least) * scale));
  };
  bool whole = false;  // all of the part, or digit, have places
  int pass = 0;
  // the bin of this pass's histogram in which the last of the `left` places falls
  auto find = [&]() -> int {
    if (warp == 0) {
      uint32_t n[8], sum = 0;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        n[e] = hist[pass & 1][255 - (8 * lane + e)];
        sum += n[e];
      }
      uint32_t before = sum;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t y = __shfl_up_sync(0xFFFFFFFFu, before, o);
        if (lane >= o) before += y;
      }
      before -= sum;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        if (before < (uint32_t)left && before + n[e] >= (uint32_t)left) {
          s_bin = 255 - (8 * lane + e);
          s_left = left - before;
          s_whole = before + n[e] == (uint32_t)left;
        }
        before += n[e];
      }
    }
    __syncthreads();
    left = (int)s_left;
    whole = s_whole != 0;
    ++pass;
    return (int)s_bin;
  };
  const bool choose = left > 0;
  int bin = 256;
  if (choose) {
#pragma unroll 8
    for (int i = m0 + tid; i < m1; i += T) atomicAdd(&hist[0][bin_of(score[i])], 1u);
    for (int i = tid; i < 256; i += T) hist[1][i] = 0;
    __syncthreads();
    bin = find();
  }
  // bits of the pages above the part (and of those that are kept anyhow), and the candidates
  const int count = (pages + 31) / 32;
  for (int w = warp; w < count; w += warps) {
    const int i = 32 * w + lane;
    bool over = i < pages && (i < m0 || i >= m1), maybe = false;
    if (choose && i >= m0 && i < m1) {
      const int k = bin_of(score[i]);
      over = k > bin || (whole && k == bin);
      maybe = !whole && k == bin;
    }
    const unsigned bo = __ballot_sync(0xFFFFFFFFu, over), bm = __ballot_sync(0xFFFFFFFFu, maybe);
    uint32_t at = 0;
    if (lane == 0) {
      words[w] = {bo, 0};
      if (bm) at = atomicAdd(&s_cand, (uint32_t)__popc(bm));
    }
    if (bm) {
      at = __shfl_sync(0xFFFFFFFFu, at, 0);
      at += __popc(bm & ((1u << lane) - 1));
      if (maybe && at < kCandidates) cand[at] = (uint16_t)i;
    }
  }
  __syncthreads();
  const int n = (int)s_cand;
  if (n > 0 && n <= kCandidates) {
    // a candidate has a place if fewer than `left` come before it
    for (int i = tid; i < n; i += T) {
      const int at = cand[i];
      const uint32_t k = score_key(score[at]);
      int before = 0;
      for (int c = 0; c < n; ++c) {
        const int other = cand[c];
        const uint32_t y = score_key(score[other]);
        before += y > k || (y == k && other < at);
      }
      if (before < left) atomicOr(&words[at >> 5].over, 1u << (at & 31));
    }
    __syncthreads();
  } else if (n > 0) {
    const int part = bin;
    uint32_t prefix = 0;
    int high = 32;
    whole = false;
    while (high > 0 && !whole) {
      const int low = high - 8;
      const uint32_t mask = high == 32 ? 0 : ~0u << high;
      for (int i = m0 + tid; i < m1; i += T) {
        const uint32_t k = score_key(score[i]);
        if (bin_of(score[i]) == part && ((k ^ prefix) & mask) == 0) atomicAdd(&hist[pass & 1][(k >> low) & 255u], 1u);
      }
      for (int i = tid; i < 256; i += T) hist[(pass & 1) ^ 1][i] = 0;
      __syncthreads();
      prefix |= (uint32_t)find() << low;
      high = low;
    }
    for (int at = m0 + tid; at < m1; at += T) {
      if (bin_of(score[at]) != part) continue;
      const uint32_t k = score_key(score[at]);
      if (whole ? k >= prefix : k > prefix) atomicOr(&words[at >> 5].over, 1u << (at & 31));
      else if (!whole && k == prefix) atomicOr(&words[at >> 5].tie, 1u << (at & 31));
    }
    __syncthreads();
  }
  // a lane per word, each warp a run of them; of the ties the first `left`
  const int run = (count + T - 1) / T * 32, w0 = warp * run;
  int n_over = 0, n_tie = 0;
  for (int w = w0 + lane; w < min(count, w0 + run); w += 32) n_over += __popc(words[w].over), n_tie += __popc(words[w].tie);
  n_over = __reduce_add_sync(0xFFFFFFFFu, n_over);
  n_tie = __reduce_add_sync(0xFFFFFFFFu, n_tie);
  if (lane == 0) above[warp] = n_over, equal[warp] = n_tie;
  __syncthreads();
  int base = __reduce_add_sync(0xFFFFFFFFu, lane < warp ? above[lane] : 0);
  int ties = __reduce_add_sync(0xFFFFFFFFu, lane < warp ? equal[lane] : 0);
  for (int w = w0; w < min(count, w0 + run); w += 32) {
    SelectWords mine{0, 0};
    if (w + lane < count) mine = words[w + lane];
    int o = __popc(mine.over), t = __popc(mine.tie);
    const int my_o = o, my_t = t;
#pragma unroll
    for (int k = 1; k < 32; k <<= 1) {
      const int y = __shfl_up_sync(0xFFFFFFFFu, o, k), z = __shfl_up_sync(0xFFFFFFFFu, t, k);
      if (lane >= k) o += y, t += z;
    }
    int at = base + o - my_o, tie = ties + t - my_t;  // chosen pages and ties before this word
    at += min(tie, left);
    for (uint32_t rest = mine.over | mine.tie; rest; rest &= rest - 1) {
      const int bit = __ffs((int)rest) - 1;
      const bool is_tie = (mine.tie >> bit) & 1;
      if (!is_tie || tie < left) out[at++] = 32 * (w + lane) + bit;
      tie += is_tie;
    }
    base += __shfl_sync(0xFFFFFFFFu, o, 31);
    ties += __shfl_sync(0xFFFFFFFFu, t, 31);
  }
}

// Lets a kernel have up to `smem` bytes of shared memory, once per device.
template <int WHICH>
cudaError_t allow_smem(const void *kern, size_t smem) {
  static std::atomic<bool> attr[64];
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev >= 0 && dev < 64 && attr[dev].load()) return cudaSuccess;
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e == cudaSuccess && dev >= 0 && dev < 64) attr[dev].store(true);
  return e;
}

}  // namespace

cudaError_t launch_page_bounds(sv_dtype dt, BoundParams p, int B, int num_sms, cudaStream_t s) {
  // Three CTAs per SM; twice as many, for sequences of different lengths, those without a page leave at
  // once.  (Six times: 16 prompts of 20000 to 32768 tokens 143.8 us, 256 sequences with 5 new tokens 5.1; three
  // times 196 and 4.0, twelve times 140.7 and 6.9.)
  const long long most = ((long long)p.cap + p.page_size - 1) / p.page_size * p.vecs;
  const long long per = std::max(1ll, std::min((most + kBoundThreads - 1) / kBoundThreads, ((long long)6 * num_sms + B - 1) / B));
  const dim3 grid((unsigned)per, (unsigned)B);
  constexpr size_t smem = 2 * kBoundRows * kBoundThreads * 16;
  const cudaError_t e = dt == SV_F32 ? allow_smem<0>((const void *)page_bounds_kernel<true>, smem) : allow_smem<1>((const void *)page_bounds_kernel<false>, smem);
  if (e != cudaSuccess) return e;
  return dt == SV_F32 ? launch_close(page_bounds_kernel<true>, grid, kBoundThreads, smem, s, p)
                      : launch_close(page_bounds_kernel<false>, grid, kBoundThreads, smem, s, p);
}

cudaError_t launch_page_scores_f32(int D, ScoreParams p, int num_sms, cudaStream_t s) {
  p.splits = std::max(1, std::min((p.P + 7) / 8, (8 * num_sms + p.units - 1) / p.units));
  return D == 128 ? launch_close(page_scores_f32_kernel<128>, dim3((unsigned)p.units * p.splits), 256, 0, s, p)
                  : launch_close(page_scores_f32_kernel<64>, dim3((unsigned)p.units * p.splits), 256, 0, s, p);
}

cudaError_t launch_select_pages(const SelectParams &p, long long lists, int num_sms, cudaStream_t s) {
  auto bytes = [](int P) { return (size_t)(P + 31) / 32 * 8 + (size_t)P * 4; };
  if (bytes(p.P) > 44 * 1024) {  // (with the kernel's other 3.6 KB more than the default 48)
    const cudaError_t e = allow_smem<2>((const void *)select_pages_kernel, bytes(SV_MAX_SCORE_PAGES));
    if (e != cudaSuccess) return e;
  }
  const int threads = p.P <= 256 ? 64 : lists <= num_sms || p.P > 8192 ? kSelectThreads : 96;
  return launch_close(select_pages_kernel, dim3((unsigned)lists), threads, bytes(p.P), s, p);
}

}  // namespace sv
