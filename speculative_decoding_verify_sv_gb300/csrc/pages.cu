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

// A CTA per list.  The threshold is found by digits of 8 bits of the keys, from the highest bit in which they
// differ at all, until the keys of the digit fill the places that are left (with random scores after two or
// three digits, of up to four); what is above it and, of those equal to it, the first ones go out in order,
// each warp a run of neighbouring pages.
__global__ void __launch_bounds__(1024) select_pages_kernel(const __grid_constant__ SelectParams p) {
  extern __shared__ uint32_t sel_smem[];
  uint32_t *keys = sel_smem;                      // [P]
  __shared__ uint32_t hist[2][256], red[2][32], s_prefix, s_left, s_full;
  __shared__ int above[32], equal[32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, T = blockDim.x, warps = T >> 5;
  const long long list = blockIdx.x;
  const int b = (int)(list / p.lists);
  for (int i = tid; i < 256; i += T) hist[0][i] = 0;
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
  uint32_t any = 0, all = 0xFFFFFFFFu;
#pragma unroll 8
  for (int i = m0 + tid; i < m1; i += T) {
    const uint32_t k = score_key(x[i]);
    keys[i] = k;
    any |= k;
    all &= k;
  }
  any = __reduce_or_sync(0xFFFFFFFFu, any);
  all = __reduce_and_sync(0xFFFFFFFFu, all);
  if (lane == 0) red[0][warp] = any, red[1][warp] = all;
  __syncthreads();
  any = __reduce_or_sync(0xFFFFFFFFu, lane < warps ? red[0][lane] : 0);
  all = __reduce_and_sync(0xFFFFFFFFu, lane < warps ? red[1][lane] : 0xFFFFFFFFu);
  int high = 32 - __clz((int)(any ^ all));  // bits below which the keys differ
  uint32_t prefix = high >= 32 ? 0 : (all >> high) << high;
  bool whole = false;  // every key that begins with the prefix has a place
  for (int pass = 0; high > 0 && left > 0 && !whole; ++pass) {
    const int low = max(0, high - 8), bins = 1 << (high - low);
    uint32_t *h = hist[pass & 1];
    const uint32_t mask = high >= 32 ? 0 : ~0u << high;
#pragma unroll 8
    for (int i = m0 + tid; i < m1; i += T) {
      const uint32_t k = keys[i];
      if (((k ^ prefix) & mask) == 0) atomicAdd(&h[(k >> low) & (bins - 1)], 1u);
    }
    for (int i = tid; i < 256; i += T) hist[(pass & 1) ^ 1][i] = 0;
    __syncthreads();
    if (warp == 0) {
      // bins from the top: the one in which the last place falls
      uint32_t n[8], sum = 0;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int bin = bins - 1 - (8 * lane + e);
        n[e] = bin >= 0 ? h[bin] : 0;
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
          s_prefix = prefix | (uint32_t)(bins - 1 - (8 * lane + e)) << low;
          s_left = left - before;
          s_full = before + n[e] == (uint32_t)left;
        }
        before += n[e];
      }
    }
    __syncthreads();
    prefix = s_prefix;
    left = (int)s_left;
    whole = s_full != 0;
    high = low;
  }
  // keys above `prefix` (or, with the whole digit, from it on), and the first `left` of those equal to it
  const bool choose = p.K > p.first + p.last;
  auto kind = [&](int i, bool &over, bool &tie) {
    over = i < pages && (i < m0 || i >= m1);
    tie = false;
    if (choose && i >= m0 && i < m1) {
      const uint32_t k = keys[i];
      over = whole ? k >= prefix : k > prefix;
      tie = !whole && k == prefix;
    }
  };
  const int run = ((pages + warps - 1) / warps + 31) & ~31, i0 = warp * run, i1 = min(pages, i0 + run);
  int n_over = 0, n_tie = 0;
  for (int i = i0; i < i1; i += 32) {
    bool over, tie;
    kind(i + lane, over, tie);
    n_over += __popc(__ballot_sync(0xFFFFFFFFu, over));
    n_tie += __popc(__ballot_sync(0xFFFFFFFFu, tie));
  }
  if (lane == 0) above[warp] = n_over, equal[warp] = n_tie;
  __syncthreads();
  int base = __reduce_add_sync(0xFFFFFFFFu, lane < warp ? above[lane] : 0);
  int ties = __reduce_add_sync(0xFFFFFFFFu, lane < warp ? equal[lane] : 0);
  const unsigned lt = (1u << lane) - 1;
  for (int i = i0; i < i1; i += 32) {
    bool over, tie;
    kind(i + lane, over, tie);
    const unsigned bo = __ballot_sync(0xFFFFFFFFu, over), bt = __ballot_sync(0xFFFFFFFFu, tie);
    const int my_ties = ties + __popc(bt & lt);
    if (over || (tie && my_ties < left)) out[base + __popc(bo & lt) + min(my_ties, left)] = i + lane;
    base += __popc(bo);
    ties += __popc(bt);
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
  const size_t smem = (size_t)p.P * 4;
  if (smem > 44 * 1024) {  // (with the kernel's other 1.5 KB more than the default 48)
    const cudaError_t e = allow_smem<2>((const void *)select_pages_kernel, SV_MAX_SCORE_PAGES * 4);
    if (e != cudaSuccess) return e;
  }
  // (2560 lists of 128 of up to 2048 pages: 23.7 us with 128 threads, 32 with 256, 46 with 512)
  const int threads = p.P <= 256 ? 128 : lists <= num_sms || p.P > 8192 ? 512 : 128;
  return launch_close(select_pages_kernel, dim3((unsigned)lists), threads, smem, s, p);
}

}  // namespace sv
