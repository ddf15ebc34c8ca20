// Scores of pages against queries on the tensor cores (tcgen05, TMEM; sm_103a, bf16).
//
// score(page, row) = sum_d max(q_d, 0) hi_d + min(q_d, 0) lo_d is one product of matrices with an inner
// size of 2 D: pages [lo | hi] (128 of them: the MMA's rows) against query rows [q- | q+] (its columns,
// up to 256 at a time).  A page is a lane of TMEM then, so that the maximum over the rows of a set is taken
// in a thread, and a warp writes the scores of 32 neighbouring pages of a set side by side.
//
// Persistent CTAs split the (sequence, KV head, tile of 128 pages) space evenly.  Two groups of four warps bring the
// bounds (cp.async: a page of a paged cache is 512 bytes somewhere in the pool) through a ring whose stages are 64
// channels of a tile's pages, the first of them also q- and q+ whenever the sequence or head changes; one warp
// issues; four read the products, double buffered in TMEM.
//
// Bound by HBM for few rows: 16 requests, one token, 2000 pages of 8 heads of 128, 26.6 us, 4.9 TB/s, 72 % of the
// measured copy rate, of which start and end are 5 us (one group of copying warps 33.5 us, mma.sync 34, gathers
// of four pages by TMA 64: 7 bytes per clock and SM); for many by the products, which HBM's time does not hide: 26
// nodes, 64:8 heads, 208 columns per page, 37 us (one group of copying warps 43, gathers 80, mma.sync 184).
#include <algorithm>
#include <atomic>
#include <climits>
#include <cmath>

#include "sv_common.cuh"
#include "sv_internal.h"
#include "tc_primitives.cuh"

namespace sv {

namespace {

using namespace tc;

constexpr int kTile = 128;        // pages of a tile
constexpr int kCols = 256;        // query rows at a time
constexpr int kScoreThreads = 416;  // maxima, copies (two groups of four warps), issue

// ST: stages of the ring; COLS: columns of a product; NQ: buffers of query rows
template <int D, int ST, int COLS_, int NQ_>
struct ScoreLayout {
  static constexpr int KB = D / 64;
  static constexpr int STAGE = kTile * 128;  // a tile's pages, 64 channels of lo or hi
  static constexpr int COLS = COLS_;
  static constexpr int NQ = NQ_;                // [2 KB][COLS][64] each, 128-byte swizzle
  static constexpr int Q_BYTES = COLS * D * 4;
  static constexpr int OFF_RING = NQ * Q_BYTES;
  static constexpr int OFF_BAR = OFF_RING + ST * STAGE;
  // full[ST], empty[ST], q_full[NQ], q_empty[NQ], d_full[2], d_empty[2], drain
  static constexpr int OFF_ROWS = OFF_BAR + (2 * ST + 5 + 2 * NQ) * 8;  // [2][2][128] rows of the bounds of a tile's pages
  static constexpr int OFF_THERE = OFF_ROWS + 4 * kTile * 4;   // [8][4] a bit for each page that is there
  static constexpr int OFF_MISC = OFF_THERE + 8 * 16;
  static constexpr int SMEM = OFF_MISC + 16;
  static_assert(SMEM <= 227 * 1024, "shared memory");
};

// Wait for the phase of the given parity; false if it ran past the limit (then *abort is raised) or *abort was
// raised.
__device__ __forceinline__ bool score_wait(uint64_t *bar, uint32_t parity, volatile int *abort, unsigned long long limit) {
  if (mbar_try_wait(bar, parity)) return true;
  const unsigned long long t0 = global_ns();
  while (!mbar_try_wait(bar, parity)) {
    if (*abort) return false;
    if (global_ns() - t0 > limit) {
      *abort = 1;
      return false;
    }
  }
  return true;
}
__device__ __forceinline__ uint32_t low_part(uint32_t a) {  // min(., 0) of two elements, a NaN kept
  uint32_t d;
  asm("min.NaN.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(0u));
  return d;
}
__device__ __forceinline__ uint32_t high_part(uint32_t a) {
  uint32_t d;
  asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(0u));
  return d;
}
__device__ __forceinline__ float larger(float a, float b) {  // a NaN is kept
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}

// A run of tiles [t0, t1) of one sequence and KV head.
struct ScoreRun {
  int b, h, t0, t1, pages;
};
__device__ __forceinline__ bool next_run(long long &w, long long end, const ScoreParams &p, int tiles, ScoreRun &r, bool reports) {
  if (w >= end) return false;
  const int bh = (int)(w / tiles);
  r.t0 = (int)(w - (long long)bh * tiles);
  r.t1 = (int)min((long long)tiles, r.t0 + (end - w));
  w += r.t1 - r.t0;
  r.h = bh % p.Hkv;
  r.b = bh / p.Hkv;
  int L = p.prefix_len[r.b];
  const int most = (int)min((long long)INT_MAX, (long long)p.P * p.page_size);
  if (L < 0 || L > most) {
    if (reports && r.h == 0) set_status(p.status, SV_DEV_BAD_PREFIX);
    L = L < 0 ? 0 : most;
  }
  r.pages = (int)(((long long)L + p.page_size - 1) / p.page_size);
  return true;
}

template <int D, int ST, int COLS_, int NQ_>
__global__ void __launch_bounds__(kScoreThreads, 1) page_scores_tc_kernel(const __grid_constant__ ScoreParams p) {
  using Lay = ScoreLayout<D, ST, COLS_, NQ_>;
  constexpr int KB = Lay::KB, COLS = Lay::COLS, NQ = Lay::NQ;
  extern __shared__ __align__(1024) uint8_t score_tc_smem[];
  uint8_t *sm = score_tc_smem, *ring = sm + Lay::OFF_RING;
  uint64_t *full = reinterpret_cast<uint64_t *>(sm + Lay::OFF_BAR), *empty = full + ST, *q_full = empty + ST, *q_empty = q_full + NQ,
           *d_full = q_empty + NQ, *d_empty = d_full + 2, *drain = d_empty + 2;
  int *s_rows = reinterpret_cast<int *>(sm + Lay::OFF_ROWS);
  volatile uint32_t *s_there = reinterpret_cast<volatile uint32_t *>(sm + Lay::OFF_THERE);
  uint32_t *s_tmem = reinterpret_cast<uint32_t *>(sm + Lay::OFF_MISC);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(s_tmem + 1);
  const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xFFFFFFFFu, tid >> 5, 0);
  const unsigned long long limit = p.wait_ns;
  const bool layout_ok = (smem_u32(sm) & 1023u) == 0;
  if (tid == 0) {
    for (int i = 0; i < ST; ++i) {
      mbar_init(&full[i], 128);
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < NQ; ++i) {
      mbar_init(&q_full[i], 128);
      mbar_init(&q_empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&d_full[i], 1);
      mbar_init(&d_empty[i], 4);
    }
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 12) {
    tmem_alloc(s_tmem, 512);
    tmem_relinquish();
  }
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *s_tmem;
  wait_previous();
  const int tiles = (p.P + kTile - 1) / kTile, cols = p.sets * p.set_cols;
  const long long total = (long long)p.units * tiles;
  long long w = total * blockIdx.x / gridDim.x;
  const long long end = layout_ok ? total * (blockIdx.x + 1) / gridDim.x : w;
  ScoreRun run;

  if (warp >= 4 && warp < 12) {
    // ------------------------------------------------------------------ copies
    // two groups of four warps, which take turns at the stages (with one of them 33.5 us against 27.2 for
    // one token of 16 sequences of 2000 pages); the first brings the query rows
    const int me = tid & 127, group = (warp - 4) >> 2;
    int k = 0, arrived = 0, segments = 0, tile = 0;  // this group's stages asked for, and landed; row chunks; tiles
    bool ok = true;
    // stages up to `upto` (of those asked for) have landed when `left` younger ones may be on their way
    auto land = [&](int upto) {
      for (; arrived < upto; ++arrived) {
        fence_proxy_async_smem();
        mbar_arrive(&full[(2 * arrived + group) % ST]);
      }
    };
    // (A wait that gives up ends the copies but not the walk, whose barriers all four warps have to reach.)
    while (next_run(w, end, p, tiles, run, false)) {
      const int t1 = min(run.t1, (run.pages + kTile - 1) / kTile);
      if (run.t0 >= t1) continue;
      for (int c0 = 0; c0 < cols; c0 += COLS) {
        // query rows of this chunk: q- and q+, each column block of 64 in rows of 128 bytes
        const int n16 = (min(COLS, cols - c0) + 15) & ~15, rows = p.set_nodes * p.G;
        const int qb = segments % NQ, q_par = (segments / NQ - 1) & 1;
        if (group == 0 && segments >= NQ && !mbar_test(&q_empty[qb], q_par)) {
          // (what is asked for lands before the products with the buffer's last rows are awaited)
          cp_async_wait<0>();
          land(k);
          ok = ok && score_wait(&q_empty[qb], q_par, abort_flag, limit);
        }
        constexpr int PER = D / 8, AT_ONCE = 8;
        const int d = me % PER;
        uint8_t *to = sm + qb * Lay::Q_BYTES + (d >> 3) * (COLS * 128);
        for (int q0 = me / PER; group == 0 && ok && q0 < n16; q0 += AT_ONCE * (128 / PER)) {
          uint4 x[AT_ONCE];
#pragma unroll
          for (int i = 0; i < AT_ONCE; ++i) {
            const int col = min(c0 + q0 + i * (128 / PER), cols - 1);
            const int set = p.sets == 1 ? 0 : col / p.set_cols, at = min(col - set * p.set_cols, rows - 1), node = at / p.G;
            x[i] = *reinterpret_cast<const uint4 *>(static_cast<const bf16 *>(p.q) +
                                                   ((((size_t)run.b * p.N + set * p.set_nodes + node) * p.Hq + run.h * p.G + at - node * p.G) * D + 8 * d));
          }
#pragma unroll
          for (int i = 0; i < AT_ONCE; ++i) {
            const int c = q0 + i * (128 / PER);
            if (c >= n16) break;
            uint8_t *at = to + sw128_offset(c, d & 7);
            *reinterpret_cast<uint4 *>(at) = make_uint4(low_part(x[i].x), low_part(x[i].y), low_part(x[i].z), low_part(x[i].w));
            *reinterpret_cast<uint4 *>(at + KB * (COLS * 128)) = make_uint4(high_part(x[i].x), high_part(x[i].y), high_part(x[i].z), high_part(x[i].w));
          }
        }
        fence_proxy_async_smem();
        if (group == 0 && ok) mbar_arrive(&q_full[qb]);
        ++segments;
        // this thread's page of a tile: its row of the bounds, read a tile ahead and looked at only then
        auto row_of = [&](int t) -> int {
          const int page = t * kTile + me;
          if (t >= t1 || page >= run.pages) return -1;
          return p.block_table ? p.block_table[(size_t)run.b * p.P + page] : run.b * p.P + page;
        };
        int next = row_of(run.t0);
        for (int t = run.t0; t < t1; ++t, ++tile) {
          int row = next;
          next = row_of(t + 1);
          if (p.block_table && (row < 0 || row >= p.num_blocks)) {
            if (group == 0 && run.h == 0 && t * kTile + me < run.pages) set_status(p.status, SV_DEV_BAD_BLOCK);
            row = -1;
          }
          int *s_row = s_rows + (2 * group + (tile & 1)) * kTile;
          const unsigned there = __ballot_sync(0xFFFFFFFFu, row >= 0);
          s_row[me] = row;
          if (group == 0 && lane == 0) s_there[(tile & 7) * 4 + warp - 4] = there;
          asm volatile("bar.sync %0, 128;" ::"r"(1 + group) : "memory");
          for (int part = group; part < 2 * KB; part += 2) {
            const int at_k = 2 * k + group, st = at_k % ST;
            ok = ok && (at_k < ST || score_wait(&empty[st], (at_k / ST - 1) & 1, abort_flag, limit));
            if (!ok) break;
            // 16-byte piece c of each 16th page
            uint8_t *dst = ring + st * Lay::STAGE;
            const int c = me & 7;
            const bf16 *src = static_cast<const bf16 *>(p.bounds) + (size_t)run.h * 2 * D + part * 64 + 8 * c;
#pragma unroll
            for (int i = 0; i < kTile / 16; ++i) {
              const int q = i * 16 + (me >> 3), at = s_row[q];
              cp_async_16(dst + sw128_offset(q, c), src + (size_t)max(at, 0) * ((size_t)p.Hkv * 2 * D), at >= 0);
            }
            cp_async_commit();
            ++k;
            cp_async_wait<ST / 2 - 1>();
            land(k - (ST / 2 - 1));
          }
          __syncwarp();
        }
      }
    }
    cp_async_wait<0>();
    land(k);
  } else if (warp == 12) {
    // ------------------------------------------------------------------- issue
    auto uniform = [](int v) { return __shfl_sync(0xFFFFFFFFu, v, 0); };
    auto arrived = [&](uint64_t *bar, int parity) -> bool { return __all_sync(0xFFFFFFFFu, score_wait(bar, parity, abort_flag, limit)); };
    auto commit = [&](uint64_t *bar) {
      if (elect_one()) umma_commit(bar);
      __syncwarp();
    };
    const uint32_t tm = __shfl_sync(0xFFFFFFFFu, tmem, 0);
    const uint64_t dq = sdesc_sw128(smem_u32(sm), 16, 1024), da = sdesc_sw128(smem_u32(ring), 16, 1024);
    int segments = 0, tile = 0, st = 0, par = 0;
    bool ok = true;
    while (ok && uniform(next_run(w, end, p, tiles, run, false))) {
      const int t0 = uniform(run.t0), t1 = uniform(min(run.t1, (run.pages + kTile - 1) / kTile));
      if (t0 >= t1) continue;
      for (int c0 = 0; ok && c0 < cols; c0 += COLS) {
        const int n16 = uniform((min(COLS, cols - c0) + 15) & ~15);
        const uint32_t id = idesc_bf16(kTile, 0, 0, 0) | (uint32_t)(n16 >> 3) << 17;
        const int qb = segments % NQ;
        ok = arrived(&q_full[qb], segments / NQ & 1);
        ++segments;
        for (int t = t0; ok && t < t1; ++t, ++tile) {
          const int buf = tile & 1;
          ok = tile < 2 || arrived(&d_empty[buf], (tile / 2 - 1) & 1);
          for (int part = 0; ok && part < 2 * KB; ++part) {
            ok = arrived(&full[st], par);
            if (!ok) break;
            tc_fence_after();
            const uint64_t a = da + (uint64_t)(st * (Lay::STAGE >> 4)), q = dq + (uint64_t)((qb * Lay::Q_BYTES + part * (COLS * 128)) >> 4);
            if (elect_one()) {
#pragma unroll
              for (int k = 0; k < 4; ++k)
                umma_bf16(tm + buf * kCols, a + (uint64_t)(k * 32 >> 4), q + (uint64_t)(k * 32 >> 4), id, part > 0 || k > 0);
              umma_commit(&empty[st]);
            }
            __syncwarp();
            if (++st == ST) st = 0, par ^= 1;
          }
          if (ok) commit(&d_full[buf]);
        }
        commit(&q_empty[qb]);
      }
    }
    commit(drain);
    const unsigned long long t0 = global_ns();
    while (!mbar_try_wait(drain, 0) && global_ns() - t0 < kWaitLimitNs) {
    }
  } else if (warp < 4) {
    // -------------------------------------------------------------- maxima, out
    int tile = 0;
    bool ok = true;
    while (ok && next_run(w, end, p, tiles, run, tid == 0)) {
      float *out = p.out + (size_t)run.b * p.sets * p.Hkv * p.P + (size_t)run.h * p.P;  // [sets][.][P]
      const size_t set_stride = (size_t)p.Hkv * p.P;
      const int t1 = min(run.t1, (run.pages + kTile - 1) / kTile);
      for (int t = max(run.t0, t1); t < run.t1; ++t) {  // tiles behind the prefix
        const int page = t * kTile + tid;
        if (page < p.P)
          for (int set = 0; set < p.sets; ++set) out[set * set_stride + page] = -INFINITY;
      }
      for (int c0 = 0; ok && run.t0 < t1 && c0 < cols; c0 += COLS) {
        const int n = min(COLS, cols - c0), n16 = (n + 15) & ~15;
        for (int t = run.t0; t < t1; ++t, ++tile) {
          const int buf = tile & 1, page = t * kTile + tid;
          if (!__all_sync(0xFFFFFFFFu, score_wait(&d_full[buf], (tile / 2) & 1, abort_flag, limit))) {
            ok = false;
            break;
          }
          tc_fence_after();
          const bool there = (s_there[(tile & 7) * 4 + warp] >> lane) & 1, inside = page < p.P;
          float best = -INFINITY;
          auto put = [&](int set, float x) {
            if (inside && set < p.sets) out[set * set_stride + page] = there ? x : -INFINITY;
          };
          for (int c = 0; c < n; c += 32) {
            float v[32];
            tmem_ld32(tmem + ((uint32_t)(warp * 32) << 16) + buf * kCols + c, v);
            tmem_wait_ld();
            const int col = c0 + c;
            if (p.sets == 1) {
              // (columns past the rows are copies of the last one up to a multiple of 16)
              if (c + 32 > n16) {
#pragma unroll
                for (int i = 16; i < 32; ++i) v[i] = v[i - 16];
              }
#pragma unroll
              for (int w8 = 16; w8 > 0; w8 >>= 1)
#pragma unroll
                for (int i = 0; i < w8; ++i) v[i] = larger(v[i], v[i + w8]);
              best = larger(best, v[0]);
              continue;
            }
            if (p.set_cols == 1) {
#pragma unroll
              for (int i = 0; i < 32; ++i)
                if (c + i < n) put(col + i, v[i]);
              continue;
            }
#pragma unroll
            for (int i = 0; i < 16; ++i) v[i] = larger(v[2 * i], v[2 * i + 1]);
            if (p.set_cols == 2) {
#pragma unroll
              for (int i = 0; i < 16; ++i)
                if (c + 2 * i < n) put(col / 2 + i, v[i]);
              continue;
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = larger(v[2 * i], v[2 * i + 1]);
            if (p.set_cols == 4) {
#pragma unroll
              for (int i = 0; i < 8; ++i)
                if (c + 4 * i < n) put(col / 4 + i, v[i]);
              continue;
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              if (c + 8 * i >= n) break;
              best = larger(best, larger(v[2 * i], v[2 * i + 1]));
              const int at = col + 8 * i, set = at / p.set_cols;
              if ((at + 8) % p.set_cols == 0 || c + 8 * i + 8 >= n) {
                // (a set whose rows came in parts: the best so far is in memory)
                if (set * p.set_cols < c0 && inside) best = larger(best, out[set * set_stride + page]);
                put(set, best);
                best = -INFINITY;
              }
            }
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&d_empty[buf]);
          if (p.sets == 1) {
            // (of more rows than a product has columns the best so far is in memory)
            if (c0 > 0 && inside) best = larger(best, out[page]);
            put(0, best);
          }
        }
      }
    }
  }
  __syncthreads();
  if (warp == 12) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
  if (tid == 0) {
    if (!layout_ok) set_status(p.status, SV_DEV_LAYOUT);
    else if (*abort_flag) set_status(p.status, SV_DEV_TIMEOUT);
  }
}

template <int D, int ST, int COLS, int NQ>
cudaError_t launch_typed(const ScoreParams &p, int grid, cudaStream_t s) {
  using Lay = ScoreLayout<D, ST, COLS, NQ>;
  static std::atomic<bool> attr[64];
  int dev = 0;
  cudaGetDevice(&dev);
  auto kern = page_scores_tc_kernel<D, ST, COLS, NQ>;
  if (dev < 0 || dev >= 64 || !attr[dev].load()) {
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Lay::SMEM);
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < 64) attr[dev].store(true);
  }
  return launch_close(kern, dim3((unsigned)grid), kScoreThreads, (size_t)Lay::SMEM, s, p);
}

// The columns of a product are query rows: those of a set one after another, padded (with the set's last
// row again, which changes no maximum) so that sets of up to 8 fill a power of two and larger ones whole
// steps of 8.
int set_columns(int rows) {
  if (rows >= 8) return (rows + 7) & ~7;
  return rows <= 1 ? 1 : rows <= 2 ? 2 : rows <= 4 ? 4 : 8;
}

}  // namespace

// A tile of 128 pages costs the same however few of them there are.  As fitted to measurements (us, heads of 64 and
// 128, 1 to 128 pages of 1 to 256 sequences): this kernel 4.6 and 2.6 per tile of an SM, the other one 0.65 for a
// thousand steps of eight rows and a page, and 1.2 for each of a set's.  E.g. one token, 32:8 heads, 64 sequences:
// 4 pages 13.2 here against 3.5, 16 pages 13.2 against 7.6, 64 pages 13.2 against 25; a set for each of 26 nodes
// of 8 heads: 8 sequences of 4 pages 9.8 against 6.0, of 16 9.8 against 17.5.
bool page_scores_prefer_tc(const ScoreParams &p, int num_sms) {
  const double cols = (double)p.sets * set_columns(p.set_nodes * p.G);
  const double tiles = std::ceil((double)p.units * ((p.P + kTile - 1) / kTile) / num_sms);
  const double here = 2.0 + 2.6 * tiles + 0.016 * cols * tiles;
  const double steps = (p.set_nodes * p.G + 7) / 8, all = 1e-3 * p.units * p.P * p.sets * steps * 152 / num_sms;
  return here <= 2.2 + std::max(1.2 * steps, 0.65 * all);
}

cudaError_t launch_page_scores_tc(int D, ScoreParams p, int num_sms, cudaStream_t s) {
  p.set_cols = set_columns(p.set_nodes * p.G);
  const long long tiles = (long long)p.units * ((p.P + kTile - 1) / kTile);
  const int grid = (int)std::min<long long>(num_sms, tiles);
  // Two buffers of query rows where there is room for them, so that a sequence or head can be prepared beside the one
  // before it, then stages: 26 nodes, 64:8 heads of 64, 16 sequences of 2048 pages 21.4 us against 28.2 with one
  // buffer (and 31.0 with one and ten stages), 64 sequences of 200 pages 21.7 against 40.7; 32:8 heads of 128,
  // 104 columns, 29.9 against 31.1; one token, 32:8 heads of 128, ten stages 26.5 against six 27.2.
  const long long cols = (long long)p.sets * p.set_cols;
  if (D == 64) return cols <= 128 ? launch_typed<64, 10, 128, 2>(p, grid, s) : launch_typed<64, 6, 256, 2>(p, grid, s);
  if (cols <= 64) return launch_typed<128, 10, 64, 2>(p, grid, s);
  return cols <= 128 ? launch_typed<128, 6, 128, 2>(p, grid, s) : launch_typed<128, 6, 256, 1>(p, grid, s);
}

}  // namespace sv
