// Block tables and slot maps from request lengths (sm_103a).
//
// A paged cache grows by pages: request b holds pages for its first length[b] tokens and is
// about to get new_tokens[b] more.  It needs
//   need_b = ceil((length_b + new_b) / bs) - ceil(length_b / bs)
// fresh pages, taken from the free list in request order (an exclusive sum over need), and its
// new token i lands in cache row table[b][p / bs] * bs + p % bs, p = length_b + i, at place
// start_b + i of the flat slot map (an exclusive sum over new).
//
// One launch, no workspace: every CTA makes both sums over the whole batch itself (8 bytes per
// request from L2, one block-wide scan) and then fills its share of the slot map, four
// neighbouring tokens per thread, so nothing is handed from CTA to CTA.  A fresh page starts
// with a new token (its first position is not below length_b), so the thread that holds this
// token writes the page's table entry.  What bounds it: 8 bytes written per token (slot and
// position); small batches are a chain of three dependent memory round trips (lengths, then a
// page id, then the stores).
#include <atomic>

#include "sv_common.cuh"
#include "sv_internal.h"

namespace sv {

namespace {

constexpr int kTableThreads = 512;
constexpr int kTableTokens = 4;  // neighbouring tokens per thread and step

// n / block_size for 0 <= n < 2^31 by a multiplication (T. Granlund, P. Montgomery, "Division by
// invariant integers using multiplication", 1994).
__device__ __forceinline__ int page_of(const TableParams &p, int n) {
  return (int)((__umulhi(p.div_mul, (unsigned)n) + (unsigned)n) >> p.div_shift);
}
__device__ __forceinline__ int pages_of(const TableParams &p, int n) { return n > 0 ? page_of(p, n - 1) + 1 : 0; }

__global__ void __launch_bounds__(kTableThreads) block_tables_kernel(const __grid_constant__ TableParams p) {
  extern __shared__ int table_smem[];
  int *s_start = table_smem;             // [B + 1] first token of each request, at most INT32_MAX
  int *s_base = table_smem + p.B + 1;    // [B] fresh pages before each request
  int *s_len = table_smem + 2 * p.B + 1; // [B] tokens that it has
  __shared__ long long s_tok[kTableThreads / 32], s_page[kTableThreads / 32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const bool report = blockIdx.x == 0;
  const long long head = p.free_head ? *p.free_head : 0;

  for (int b = tid; b < p.B; b += kTableThreads) {
    int L = __ldg(p.length + b), x = __ldg(p.new_tokens + b);
    if (report && (L < 0 || L > p.cap || x < 0 || x > p.cap - L)) set_status(p.status, SV_DEV_BAD_PREFIX);
    L = L < 0 ? 0 : min(L, p.cap);
    // (tokens past the table get no slot; more of them than the slot map has room for count as
    // that many, so that a wild number does not make a long loop)
    x = x < 0 ? 0 : (int)min((long long)x, min((long long)p.cap - L + p.T, (long long)INT32_MAX - L));
    s_start[b] = x;
    s_base[b] = max(0, min(pages_of(p, L + x), p.max_blocks) - pages_of(p, L));
    s_len[b] = L;
  }
  __syncthreads();
  // each thread sums a run of requests (an odd run length: no bank conflicts), then the runs
  const int per = ((p.B + kTableThreads - 1) / kTableThreads) | 1;
  const int b0 = min(tid * per, p.B), b1 = min(b0 + per, p.B);
  long long tok = 0, page = 0;
  for (int b = b0; b < b1; ++b) {
    tok += s_start[b];
    page += s_base[b];
  }
  long long itok = tok, ipage = page;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long yt = __shfl_up_sync(0xFFFFFFFFu, itok, o), yp = __shfl_up_sync(0xFFFFFFFFu, ipage, o);
    if (lane >= o) {
      itok += yt;
      ipage += yp;
    }
  }
  if (lane == 31) {
    s_tok[warp] = itok;
    s_page[warp] = ipage;
  }
  __syncthreads();
  long long total = 0, pages = 0, btok = 0, bpage = 0;
#pragma unroll
  for (int w = 0; w < kTableThreads / 32; ++w) {
    if (w == warp) {
      btok = total;
      bpage = pages;
    }
    total += s_tok[w];
    pages += s_page[w];
  }
  btok += itok - tok;
  bpage += ipage - page;
  for (int b = b0; b < b1; ++b) {
    const int n = s_start[b], need = s_base[b];
    s_start[b] = (int)min(btok, (long long)INT32_MAX);
    s_base[b] = (int)min(bpage, (long long)INT32_MAX);
    btok += n;
    bpage += need;
  }
  if (tid == 0) s_start[p.B] = (int)min(total, (long long)INT32_MAX);
  __syncthreads();

  if (report) {
    for (int b = tid; b <= p.B; b += kTableThreads) p.token_start[b] = s_start[b];
    if (tid == 0) {
      p.out_free_head[0] = (int)min(head + pages, (long long)INT32_MAX);
      if (total > p.T) set_status(p.status, SV_DEV_BAD_PREFIX);
      if (head < 0 || (pages > 0 && head + pages > p.num_free)) set_status(p.status, SV_DEV_BAD_BLOCK);
    }
  }

  // tokens in steps of four per thread over all CTAs: up to the batch's last (its pages are
  // given out even where the slot map is too short) and on to the end of the slot map
  const long long end = max(total, (long long)p.T);
  const long long step = (long long)gridDim.x * kTableThreads * kTableTokens;
  for (long long t0 = ((long long)blockIdx.x * kTableThreads + tid) * kTableTokens; t0 < end; t0 += step) {
    int slot[kTableTokens], pos[kTableTokens];
    int b = -1, have = 0, pg = -1, off = 0, row = -1, stop = 0;
    long long fresh = 0;
#pragma unroll
    for (int k = 0; k < kTableTokens; ++k) {
      const long long t = t0 + k;
      slot[k] = pos[k] = -1;
      if (t >= total || t >= INT32_MAX) continue;
      bool look = false;  // the page's id has to be read
      if (b < 0 || t >= stop) {
        // the last request that starts at or before t (the ones without tokens are passed over)
        int lo = b < 0 ? 0 : b, hi = p.B;  // start[lo] <= t < start[hi]
        while (hi - lo > 1) {
          const int mid = (lo + hi) >> 1;
          if (s_start[mid] <= t) lo = mid;
          else hi = mid;
        }
        b = lo;
        stop = s_start[b + 1];
        const int len = s_len[b];
        have = pages_of(p, len);
        pos[k] = len + (int)(t - s_start[b]);
        pg = page_of(p, pos[k]);
        off = pos[k] - pg * p.block_size;
        fresh = head + s_base[b] - have;
        look = true;
      } else {
        pos[k] = pos[k > 0 ? k - 1 : 0] + 1;
        if (++off == p.block_size) {
          off = 0;
          ++pg;
          look = true;
        }
      }
      if (look) {
        row = -1;
        if (pg < p.max_blocks) {
          int32_t *entry = p.block_table + (size_t)b * p.max_blocks + pg;
          if (pg < have) {
            row = *entry;
          } else {
            const long long i = fresh + pg;
            if (i >= 0 && i < p.num_free && head >= 0) row = __ldg(p.free_blocks + i);
          }
          if (row < 0 || row >= p.num_blocks) {
            set_status(p.status, SV_DEV_BAD_BLOCK);
            row = -1;
          }
          if (pg >= have && off == 0) *entry = row;
        }
      }
      if (row >= 0) slot[k] = row * p.block_size + off;
    }
    if (t0 + kTableTokens <= p.T) {
      *reinterpret_cast<int4 *>(p.slots + t0) = make_int4(slot[0], slot[1], slot[2], slot[3]);
      *reinterpret_cast<int4 *>(p.positions + t0) = make_int4(pos[0], pos[1], pos[2], pos[3]);
    } else {
#pragma unroll
      for (int k = 0; k < kTableTokens; ++k)
        if (t0 + k < p.T) {
          p.slots[t0 + k] = slot[k];
          p.positions[t0 + k] = pos[k];
        }
    }
  }
}

}  // namespace

cudaError_t launch_block_tables(TableParams p, int num_sms, cudaStream_t s) {
  const long long cap = (long long)p.max_blocks * p.block_size;
  p.cap = (int)(cap < INT32_MAX ? cap : INT32_MAX);
  p.div_shift = 0;
  while ((1ll << p.div_shift) < p.block_size) ++p.div_shift;
  p.div_mul = (unsigned)(((1ull << 32) * ((1ull << p.div_shift) - p.block_size)) / p.block_size + 1);
  const size_t smem = (size_t)(3 * p.B + 1) * sizeof(int);
  static std::atomic<bool> attr_set[64];
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev < 0 || dev >= 64 || !attr_set[dev].load()) {
    const cudaError_t e = cudaFuncSetAttribute(block_tables_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               (int)((3 * SV_MAX_TABLE_BATCH + 1) * sizeof(int)));
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < 64) attr_set[dev].store(true);
  }
  const long long per_cta = kTableThreads * kTableTokens;
  long long ctas = (p.T + per_cta - 1) / per_cta;
  ctas = ctas < 1 ? 1 : (ctas > 2ll * num_sms ? 2ll * num_sms : ctas);
  block_tables_kernel<<<(unsigned)ctas, kTableThreads, smem, s>>>(p);
  return cudaGetLastError();
}

}  // namespace sv
