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
  const int first = start / p.page_size, pages = (int)(((long long)L + p.page_size - 1) / p.page_size) - first;
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

// ------------------------------------------ scores without the tensor cores (page_scores_tc.cu: with)

// A warp per page and set, a lane's channels next to one another.  Eight rows are summed over the lanes together: each
// exchange halves the rows of a lane.  For fp32, and for bf16 where a tile of 128 pages would be mostly
// empty (page_scores_prefer_tc).
template <typename T, int D>
__global__ void __launch_bounds__(256) page_scores_plain_kernel(const __grid_constant__ ScoreParams p) {
  constexpr int PL = D / 32;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int bh = blockIdx.x / p.splits, part = blockIdx.x % p.splits, h = bh % p.Hkv, b = bh / p.Hkv, warps = blockDim.x >> 5;
  wait_previous();
  int L = p.prefix_len[b];
  const int most = (int)min((long long)INT_MAX, (long long)p.P * p.page_size);
  if (L < 0 || L > most) {
    if (h == 0 && part == 0 && threadIdx.x == 0) set_status(p.status, SV_DEV_BAD_PREFIX);
    L = L < 0 ? 0 : most;
  }
  const int pages = (int)(((long long)L + p.page_size - 1) / p.page_size);
  float *out = p.out + (size_t)b * p.sets * p.Hkv * p.P + (size_t)h * p.P;
  // PL neighbouring elements
  struct alignas(sizeof(T) * PL) Piece {
    T x[PL];
  };
  const int rows = p.set_nodes * p.G;
  const long long jobs = (long long)p.P * p.sets;
  for (long long job = (long long)part * warps + warp; job < jobs; job += (long long)p.splits * warps) {
    const int set = (int)(job / p.P), page = (int)(job - (long long)set * p.P);
    long long row = -1;
    if (page < pages) {
      if (!p.block_table) {
        row = (long long)b * p.P + page;
      } else {
        const int blk = p.block_table[(size_t)b * p.P + page];
        if (blk >= 0 && blk < p.num_blocks) row = blk;
        else if (h == 0 && set == 0 && lane == 0) set_status(p.status, SV_DEV_BAD_BLOCK);
      }
    }
    if (row < 0) {
      if (lane == 0) out[(size_t)set * p.Hkv * p.P + page] = -INFINITY;
      continue;
    }
    const T *src = static_cast<const T *>(p.bounds) + ((size_t)row * p.Hkv + h) * 2 * D + PL * lane;
    const Piece lo = *reinterpret_cast<const Piece *>(src), hi = *reinterpret_cast<const Piece *>(src + D);
    float best = -INFINITY;  // of the rows r0 + k, a k for each four lanes
    for (int r0 = 0; r0 < rows; r0 += 8) {
      float x[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int r = min(r0 + k, rows - 1), node = r / p.G;
        const Piece q = *reinterpret_cast<const Piece *>(
            static_cast<const T *>(p.q) + (((size_t)b * p.N + set * p.set_nodes + node) * p.Hq + h * p.G + r - node * p.G) * D + PL * lane);
        x[k] = 0.f;
#pragma unroll
        for (int i = 0; i < PL; ++i) {
          const float y = (float)q.x[i];
          x[k] = fmaf(max_nan(y, 0.f), (float)hi.x[i], x[k]);
          x[k] = fmaf(min_nan(y, 0.f), (float)lo.x[i], x[k]);
        }
      }
      // (rows past the last are it once more, which changes no maximum)
#pragma unroll
      for (int half = 4; half > 0; half >>= 1) {
        const bool upper = lane & (4 * half);
#pragma unroll
        for (int k = 0; k < half; ++k) {
          const float keep = upper ? x[k + half] : x[k], send = upper ? x[k] : x[k + half];
          x[k] = keep + __shfl_xor_sync(0xFFFFFFFFu, send, 4 * half);
        }
      }
      x[0] += __shfl_xor_sync(0xFFFFFFFFu, x[0], 2);
      x[0] += __shfl_xor_sync(0xFFFFFFFFu, x[0], 1);
      best = max_nan(best, x[0]);
    }
#pragma unroll
    for (int o = 4; o < 32; o <<= 1) best = max_nan(best, __shfl_xor_sync(0xFFFFFFFFu, best, o));
    if (lane == 0) out[(size_t)set * p.Hkv * p.P + page] = best;
  }
}

// ------------------------------------------------------------------- selection

// Order-preserving key of a score: larger for larger scores, the largest for a NaN; the two zeros are one.
__device__ __forceinline__ uint32_t score_key(float x) {
  if (x != x) return 0xFFFFFFFFu;
  const uint32_t u = __float_as_uint(x + 0.f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// A list is a warp's (many lists) or a CTA's, in whose registers its scores are, up to E per thread.  One histogram
// of 256 equal parts of the scores' range gives the part in which the last place falls.  What is above it is
// chosen; what is in it are candidates, few as a rule, of which each counts those before it (or, many of them,
// digits of 8 bits of their keys decide, and of those equal to the end the lower pages).  The chosen pages are
// bits of words, which lanes hold and put out.
// Bound by instructions and their latency: 2560 lists of up to 2048 scores 15.7 us (of 17.8 before the loops ran without
// branches 3.7 started, 2.1 loaded, 3 found the parts, 2.6 counted, 4.1 sorted out, 2.3 put out); with the scores in
// shared memory, 4500 instructions per list, 18.3; the highest bits in which the keys differ as the parts, where
// scores of both signs meet in a few words, 23; without atomics, by counts against seven pivots at a time, 25.3.
constexpr int kSelectWarps = 2;  // a list each

template <int E, bool WARP>
struct SelectShared {
  static constexpr int WARPS = WARP ? 1 : E == 32 ? 32 : 16;  // of a list, at most
  static constexpr int CAND = WARP ? 128 : 512;  // candidates of a list; more of them are looked up again
  uint32_t hist[256], key[CAND], over[WARPS * E], tie[WARPS * E], bin, left, whole, count;
  uint16_t cand[CAND];
  float least[WARPS], largest[WARPS];
  int above[WARPS], equal[WARPS];
};

template <int E, bool WARP>
__global__ void __launch_bounds__(WARP ? 32 * kSelectWarps : 32 * SelectShared<E, WARP>::WARPS)
    select_pages_kernel(const __grid_constant__ SelectParams p) {
  using Shared = SelectShared<E, WARP>;
  constexpr int STEP = E < 8 ? E : 8;
  __shared__ Shared shared[WARP ? kSelectWarps : 1];
  const int lane = threadIdx.x & 31, cta_warp = __shfl_sync(0xFFFFFFFFu, (int)threadIdx.x >> 5, 0);
  const int warp = WARP ? 0 : cta_warp, tid = WARP ? lane : (int)threadIdx.x, T = WARP ? 32 : (int)blockDim.x, warps = T >> 5;
  Shared &sh = shared[WARP ? cta_warp : 0];
  auto sync = [] {
    if constexpr (WARP) __syncwarp();
    else __syncthreads();
  };
  const long long list = WARP ? (long long)blockIdx.x * kSelectWarps + cta_warp : blockIdx.x;
  const int b = (int)(list / p.lists);
  if (b >= p.B) return;
  for (int i = tid; i < 256; i += T) sh.hist[i] = 0;
  for (int i = tid; i < warps * E; i += T) sh.over[i] = sh.tie[i] = 0;
  if (tid == 0) sh.count = 0;
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
  // pages [m0, m1) compete for `left` places; this warp's words of 32 pages are [w0, w0 + n), and of this lane's
  // pages at0 + 32 e those with e in [e0, e1) compete
  const int m0 = p.first, m1 = pages - p.last, count = (pages + 31) / 32, per = (count + warps - 1) / warps;
  const int w0 = min(count, warp * per), n = min(count, w0 + per) - w0, at0 = 32 * w0 + lane;
  const int e0 = (max(m0 - at0, 0) + 31) / 32, e1 = min(n, (max(m1 - at0, 0) + 31) / 32);
  int left = p.K - p.first - p.last;
  const float *scores = p.scores + list * p.P;
  float x[E];
#pragma unroll
  for (int e = 0; e < E; ++e) x[e] = e >= e0 && e < e1 ? scores[at0 + 32 * e] : __int_as_float(0x7FC00000);
  // the least and largest finite ones
  float least[2] = {FLT_MAX, FLT_MAX}, largest[2] = {-FLT_MAX, -FLT_MAX};
#pragma unroll
  for (int e = 0; e < E; ++e) {
    least[e & 1] = fminf(least[e & 1], x[e]);
    largest[e & 1] = fmaxf(largest[e & 1], x[e]);
  }
  float lo = fminf(least[0], least[1]), hi = fmaxf(largest[0], largest[1]);
  if (lo < -FLT_MAX || hi > FLT_MAX) {
    lo = FLT_MAX, hi = -FLT_MAX;
#pragma unroll
    for (int e = 0; e < E; ++e)
      if (fabsf(x[e]) <= FLT_MAX) lo = fminf(lo, x[e]), hi = fmaxf(hi, x[e]);
  }
  auto extremes = [&] {
    asm volatile("redux.sync.min.f32 %0, %0, 0xFFFFFFFF;" : "+f"(lo));
    asm volatile("redux.sync.max.f32 %0, %0, 0xFFFFFFFF;" : "+f"(hi));
  };
  __syncwarp();
  extremes();
  if constexpr (!WARP) {
    if (lane == 0) sh.least[warp] = lo, sh.largest[warp] = hi;
    __syncthreads();
    lo = lane < warps ? sh.least[lane] : FLT_MAX;
    hi = lane < warps ? sh.largest[lane] : -FLT_MAX;
    extremes();
  }
  // Parts of the range, growing with the score; infinities and NaN are at the ends.  Without a range (equal
  // scores, no finite ones, or an overflow) there is one part.
  const float range = hi - lo, scale = range > 0.f && range <= FLT_MAX ? 255.f / range : 0.f;
  const bool one_part = !(scale > 0.f && scale <= FLT_MAX), choose = left > 0;
  int part[E];  // of each score that competes, -1 for the others
#pragma unroll
  for (int c = 0; c < E; c += STEP) {
    if (c < n) {
#pragma unroll
      for (int e = c; e < c + STEP; ++e) {
        const unsigned k = min(255u, __float2uint_rz((x[e] - lo) * scale));  // (-infinity: 0)
        part[e] = x[e] == x[e] ? (int)k : 255;
        if (one_part) part[e] = 0;
        if (e < e0 || e >= e1) part[e] = -1;
        if (choose && part[e] >= 0) atomicAdd(&sh.hist[part[e]], 1u);
      }
    } else {
#pragma unroll
      for (int e = c; e < c + STEP; ++e) part[e] = -1;
    }
  }
  // the bin of the histogram in which the last of the `left` places falls
  bool whole = false;  // all of the part, or digit, have places
  auto find = [&]() -> int {
    sync();
    if (warp == 0) {
      uint32_t m[8], sum = 0;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        m[e] = sh.hist[255 - (8 * lane + e)];
        sum += m[e];
      }
      uint32_t before = sum;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t y = __shfl_up_sync(0xFFFFFFFFu, before, o);
        if (lane >= o) before += y;
      }
      before -= sum;
      if (before < (uint32_t)left && before + sum >= (uint32_t)left) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          if (before < (uint32_t)left && before + m[e] >= (uint32_t)left) {
            sh.bin = 255 - (8 * lane + e);
            sh.left = left - before;
            sh.whole = before + m[e] == (uint32_t)left;
          }
          before += m[e];
        }
      }
    }
    sync();
    left = (int)sh.left;
    whole = sh.whole != 0;
    return (int)sh.bin;
  };
  const int last = choose ? find() : 1000;
  // this lane's word of the chosen pages, and which of its pages are candidates
  uint32_t mine = 0, maybe = 0;
  const int over_from = whole ? last : last + 1, maybe_at = whole || !choose ? 1000 : last;
#pragma unroll
  for (int c = 0; c < E; c += STEP) {
    if (c < n) {
#pragma unroll
      for (int e = c; e < c + STEP; ++e) {
        const unsigned over = __ballot_sync(0xFFFFFFFFu, part[e] >= over_from);
        if (lane == e) mine = over;
        if (part[e] == maybe_at) maybe |= 1u << e;
      }
    }
  }
  if (maybe) {
    int at = (int)atomicAdd(&sh.count, (uint32_t)__popc(maybe));
    for (uint32_t rest = maybe; rest; rest &= rest - 1, ++at) {
      const int page = at0 + 32 * (__ffs((int)rest) - 1);
      if (at < Shared::CAND) sh.cand[at] = (uint16_t)page, sh.key[at] = score_key(scores[page]);
    }
  }
  sync();
  const int candidates = (int)sh.count;
  if (candidates > 0 && candidates <= Shared::CAND) {
    // a candidate has a place if fewer than `left` come before it
    for (int i = tid; i < candidates; i += T) {
      const int at = sh.cand[i];
      const uint32_t k = sh.key[i];
      int before = 0;
      for (int c = 0; c < candidates; ++c) {
        const uint32_t y = sh.key[c];
        before += y > k || (y == k && sh.cand[c] < at);
      }
      if (before < left) atomicOr(&sh.over[at >> 5], 1u << (at & 31));
    }
    sync();
  } else if (candidates > 0) {
    uint32_t prefix = 0;
    int high = 32;
    auto each = [&](auto f) {
      for (uint32_t rest = maybe; rest; rest &= rest - 1) {
        const int page = at0 + 32 * (__ffs((int)rest) - 1);
        f(page, score_key(scores[page]));
      }
      __syncwarp();
    };
    whole = false;
#pragma unroll 1
    while (high > 0 && !whole) {
      const int low = high - 8;
      const uint32_t mask = high == 32 ? 0 : ~0u << high;
      for (int i = tid; i < 256; i += T) sh.hist[i] = 0;
      sync();
      each([&](int, uint32_t k) {
        if (((k ^ prefix) & mask) == 0) atomicAdd(&sh.hist[(k >> low) & 255u], 1u);
      });
      prefix |= (uint32_t)find() << low;
      high = low;
    }
    each([&](int page, uint32_t k) {
      if (whole ? k >= prefix : k > prefix) atomicOr(&sh.over[page >> 5], 1u << (page & 31));
      else if (!whole && k == prefix) atomicOr(&sh.tie[page >> 5], 1u << (page & 31));
    });
    sync();
  }
  // with the pages that are kept anyhow; of the ties the first `left`
  uint32_t tied = 0;
  if (lane < n) {
    const int page = 32 * (w0 + lane);
    auto below = [&](int end) { return end <= page ? 0u : end >= page + 32 ? ~0u : (1u << (end - page)) - 1; };
    mine |= sh.over[w0 + lane] | below(m0) | (below(pages) & ~below(m1));
    tied = sh.tie[w0 + lane];
  }
  int at = __popc(mine), tie = __popc(tied);  // up to this word
#pragma unroll
  for (int s = 1; s < 32; s <<= 1) {
    const int y = __shfl_up_sync(0xFFFFFFFFu, at, s), z = __shfl_up_sync(0xFFFFFFFFu, tie, s);
    if (lane >= s) at += y, tie += z;
  }
  if constexpr (!WARP) {
    if (lane == 31) sh.above[warp] = at, sh.equal[warp] = tie;
    __syncthreads();
    at += __reduce_add_sync(0xFFFFFFFFu, lane < warp ? sh.above[lane] : 0);
    tie += __reduce_add_sync(0xFFFFFFFFu, lane < warp ? sh.equal[lane] : 0);
  }
  tie -= __popc(tied);
  at += min(tie, left) - __popc(mine);
  for (uint32_t rest = mine | tied; rest; rest &= rest - 1) {
    const int bit = __ffs((int)rest) - 1;
    const bool is_tie = (tied >> bit) & 1;
    if (!is_tie || tie < left) out[at++] = 32 * (w0 + lane) + bit;
    tie += is_tie;
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

cudaError_t launch_page_scores_plain(sv_dtype dt, int D, ScoreParams p, int num_sms, cudaStream_t s) {
  const long long jobs = (long long)p.P * p.sets;
  const int warps = (int)std::min<long long>(8, jobs);
  p.splits = (int)std::max<long long>(1, std::min<long long>((jobs + warps - 1) / warps, (64ll / warps * num_sms + p.units - 1) / p.units));
  const dim3 grid((unsigned)((long long)p.units * p.splits));
  if (dt == SV_F32)
    return D == 128 ? launch_close(page_scores_plain_kernel<float, 128>, grid, 32 * warps, 0, s, p)
                    : launch_close(page_scores_plain_kernel<float, 64>, grid, 32 * warps, 0, s, p);
  return D == 128 ? launch_close(page_scores_plain_kernel<bf16, 128>, grid, 32 * warps, 0, s, p)
                  : launch_close(page_scores_plain_kernel<bf16, 64>, grid, 32 * warps, 0, s, p);
}

// Many lists (four per SM): a warp per list of up to 1024 scores, 16 scores per thread for longer ones; else few scores
// per thread.  Measured, us a warp / 16 per thread / 4 per thread, 152 SMs:
//   512 scores    152 lists 4.0 / 5.0 / 3.5;  608 lists 4.1 / 5.1 / 4.2;  2560 lists 5.7 / 7.0 / 9.1
//   1000 scores   152 lists 5.1 / 5.1 / 3.9;  608 lists 5.4 / 5.6 / 5.3;  2560 lists 8.3 / 10.9 / 15.4
//   2048 scores   152 lists 9.7 / 5.6 / 4.7;  608 lists 10.2 / 6.7 / 8.4;  2560 lists 20 / 17.1 / 28.9
cudaError_t launch_select_pages(const SelectParams &p, int num_sms, cudaStream_t s) {
  const long long lists = (long long)p.B * p.lists;
  const bool many = lists >= 4ll * num_sms;
  if (many && p.P <= 1024) {
    const dim3 grid((unsigned)((lists + kSelectWarps - 1) / kSelectWarps));
    if (p.P <= 512) return launch_close(select_pages_kernel<16, true>, grid, 32 * kSelectWarps, 0, s, p);
    return launch_close(select_pages_kernel<32, true>, grid, 32 * kSelectWarps, 0, s, p);
  }
  const int e = p.P <= 2048 && !many ? 4 : p.P <= 8192 ? 16 : 32;
  const dim3 grid((unsigned)lists);
  const int threads = (p.P + 32 * e - 1) / (32 * e) * 32;
  if (e == 4) return launch_close(select_pages_kernel<4, false>, grid, threads, 0, s, p);
  if (e == 16) return launch_close(select_pages_kernel<16, false>, grid, threads, 0, s, p);
  return launch_close(select_pages_kernel<32, false>, grid, threads, 0, s, p);
}

}  // namespace sv
