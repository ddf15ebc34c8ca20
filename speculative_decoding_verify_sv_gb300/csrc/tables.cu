// Block tables and slot maps from request lengths (sm_103a).
//
// A paged cache grows by pages: request b holds pages for its first length[b] tokens and is
// about to get new_tokens[b] more.  It needs
//   need_b = ceil((length_b + new_b) / bs) - ceil(length_b / bs)
// fresh pages, taken from the free list in request order (an exclusive sum over need), and its
// new token i lands in cache row table[b][p / bs] * bs + p % bs, p = length_b + i, at place
// start_b + i of the flat slot map (an exclusive sum over new).  A round that asked for more tokens
// than it kept leaves pages behind that its length does not reach; where the caller says how many
// pages a row holds, that number stands in the place of ceil(length_b / bs) if it is the larger.
//
// One launch, no workspace: every CTA makes both sums over the whole batch itself (8 bytes per
// request from L2, one block-wide scan) and then fills its share of the slot map, so nothing is
// handed from CTA to CTA.  A thread finds the requests of its tokens by a search of a fixed number
// of steps, several tokens side by side, so that neither the searches nor the reads of the page
// ids wait for one another.  Where requests bring many tokens (256 places of the map per request
// and more) a thread takes four neighbouring tokens, which mostly share their request and page: 256
// prompts of 512 to 8192 tokens 8.1 us (8.9 with 64-bit places) against 16.4 with single tokens; 4096
// requests of up to 64 tokens 7.3 us with single tokens against 9.9 with four, whose crossings of
// requests diverge.
// A fresh page starts with a new token (its first position is not below length_b), so the thread
// that holds this token writes the page's table entry.
// What bounds it: 8 bytes written per token (slot and position); small batches are a chain of
// three dependent memory round trips (lengths, page ids, stores) and two block barriers.
#include <algorithm>
#include <atomic>

#include "sv_common.cuh"
#include "sv_internal.h"

namespace sv {

namespace {

constexpr int kTableLoads = 4;   // requests per thread whose sizes are loaded together

// n / block_size for 0 <= n < 2^31 by a multiplication (T. Granlund, P. Montgomery, "Division by
// invariant integers using multiplication", 1994).
__device__ __forceinline__ int page_of(const TableParams &p, int n) {
  return (int)((__umulhi(p.div_mul, (unsigned)n) + (unsigned)n) >> p.div_shift);
}
__device__ __forceinline__ int pages_of(const TableParams &p, int n) { return n > 0 ? page_of(p, n - 1) + 1 : 0; }

// More tokens than the slot map has room for: the pages whose first token lies past its end are given
// out page by page (of a batch of 2^31 fresh pages and more the first 2^31 - 1), so that the time goes by
// the table's entries and not by the number of tokens, however wild.  Out of line: in the kernel's own
// code, where it is hardly ever reached, it costs every call 0.3 us.
template <bool HELD>
__device__ __noinline__ void pages_past_the_map(const TableParams &p, const int *sums, long long head, long long pages) {
  const int *s_start = sums, *s_base = sums + p.B + 1, *s_len = sums + 2 * p.B + 1, *s_have = sums + 3 * p.B + 1;
  auto pages_had = [&](int b) { return HELD ? s_have[b] : pages_of(p, s_len[b]); };
  const int top = p.B > 1 ? 1 << (31 - __clz(p.B - 1)) : 0;
  const unsigned left = head >= 0 && head < p.num_free ? (unsigned)(p.num_free - head) : 0u;
  unsigned from = 0;
  if (p.T > 0) {  // behind the pages up to the last token with a place
    int b = 0;
    for (int d = top; d > 0; d >>= 1)
      if (b + d < p.B && s_start[b + d] < p.T) b += d;
    from = (unsigned)s_base[b] +
           (unsigned)max(0, min(pages_of(p, s_len[b] + (p.T - s_start[b])), p.max_blocks) - pages_had(b));
  }
  const unsigned last = (unsigned)min(pages, (long long)INT32_MAX);
  bool bad = false;
  for (unsigned i = from + blockIdx.x * blockDim.x + threadIdx.x; i < last; i += gridDim.x * blockDim.x) {
    int b = 0;  // the last request whose fresh pages begin at or before page i
    for (int d = top; d > 0; d >>= 1)
      if (b + d < p.B && (unsigned)s_base[b + d] <= i) b += d;
    const int id = i < left ? p.free_blocks[head + i] : -1;
    const bool there = (unsigned)id < (unsigned)p.num_blocks;
    p.block_table[(size_t)b * p.max_blocks + pages_had(b) + (int)(i - (unsigned)s_base[b])] = there ? id : -1;
    if (!there) bad = true;
  }
  if (bad) set_status(p.status, SV_DEV_BAD_BLOCK);
}

// RUN: neighbouring tokens per thread (1: two tokens a block apart).  HELD: rows may hold more pages
// than those of their tokens (an instance of its own: one more array to read and keep costs up to 0.3 us, 4096 requests).
template <int RUN, int kTableThreads, bool HELD>
__global__ void __launch_bounds__(kTableThreads) block_tables_kernel(const __grid_constant__ TableParams p) {
  extern __shared__ int table_smem[];
  int *s_start = table_smem;             // [B + 1] first token of each request, at most INT32_MAX
  int *s_base = table_smem + p.B + 1;    // [B] fresh pages before each request
  int *s_len = table_smem + 2 * p.B + 1; // [B] tokens that it has
  int *s_have = table_smem + 3 * p.B + 1; // [B] pages that it has (HELD; else those of its tokens)
  __shared__ long long s_tok[kTableThreads / 32], s_page[kTableThreads / 32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const bool report = blockIdx.x == 0;
  wait_previous();
  const long long head = p.free_head ? *p.free_head : 0;

  for (int c = 0; c < p.B; c += kTableThreads * kTableLoads) {
    int len[kTableLoads], add[kTableLoads], held[kTableLoads];
#pragma unroll
    for (int k = 0; k < kTableLoads; ++k) {
      const int b = c + k * kTableThreads + tid;
      len[k] = b < p.B ? p.length[b] : 0;
      add[k] = b < p.B ? p.new_tokens[b] : 0;
      held[k] = HELD && b < p.B ? p.held[b] : 0;
    }
#pragma unroll
    for (int k = 0; k < kTableLoads; ++k) {
      const int b = c + k * kTableThreads + tid;
      if (b >= p.B) break;
      int L = len[k], x = add[k];
      if (report && (L < 0 || L > p.cap || x < 0 || x > p.cap - L)) set_status(p.status, SV_DEV_BAD_PREFIX);
      L = L < 0 ? 0 : min(L, p.cap);
      // (tokens past the table get no slot; more of them than the slot map has room for count
      // as that many)
      x = x < 0 ? 0 : (int)min((long long)x, min((long long)p.cap - L + p.T, (long long)INT32_MAX - L));
      int have = pages_of(p, L);
      if constexpr (HELD) {
        if (report && (held[k] < 0 || held[k] > p.max_blocks)) set_status(p.status, SV_DEV_BAD_PREFIX);
        s_have[b] = have = max(have, min(held[k], p.max_blocks));
      }
      s_start[b] = x;
      s_base[b] = max(0, min(pages_of(p, L + x), p.max_blocks) - have);
      s_len[b] = L;
      if (HELD && report) p.out_held[b] = have + s_base[b];
    }
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
  // every warp sums the warps' totals
  const bool mine = lane < kTableThreads / 32;
  long long wtok = mine ? s_tok[lane] : 0, wpage = mine ? s_page[lane] : 0;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long yt = __shfl_up_sync(0xFFFFFFFFu, wtok, o), yp = __shfl_up_sync(0xFFFFFFFFu, wpage, o);
    if (lane >= o) {
      wtok += yt;
      wpage += yp;
    }
  }
  const long long total = __shfl_sync(0xFFFFFFFFu, wtok, 31), pages = __shfl_sync(0xFFFFFFFFu, wpage, 31);
  long long btok = __shfl_sync(0xFFFFFFFFu, wtok, max(warp - 1, 0)), bpage = __shfl_sync(0xFFFFFFFFu, wpage, max(warp - 1, 0));
  if (warp == 0) btok = bpage = 0;
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

  // The slot map's places, 32-bit numbers; the pages of tokens past its end follow below.
  const unsigned tokens = (unsigned)min(total, (long long)p.T), end = (unsigned)p.T;
  constexpr int U = RUN == 1 ? 2 : RUN;
  const unsigned step = gridDim.x * kTableThreads * U;
  const int top = p.B > 1 ? 1 << (31 - __clz(p.B - 1)) : 0;  // the search's first stride
  auto pages_had = [&](int b) { return HELD ? s_have[b] : pages_of(p, s_len[b]); };
  // where the id of page pg of request b is: held (in the table) or fresh (NULL: none is left)
  const unsigned left = head >= 0 && head < p.num_free ? (unsigned)(p.num_free - head) : 0u;
  const int32_t *fresh = p.free_blocks + (left ? head : 0);
  auto page_source = [&](int b, int pg, int have) -> const int32_t * {
    if (pg >= p.max_blocks) return nullptr;
    if (pg < have) return p.block_table + (size_t)b * p.max_blocks + pg;
    const unsigned i = (unsigned)s_base[b] + (unsigned)(pg - have);
    return i < left ? fresh + i : nullptr;
  };
  bool bad = false;  // an id outside the pool, or none left
  // the id as it was read, checked; the entry of a fresh page is written with its first token
  auto checked = [&](int row, int b, int pg, bool entry) -> int {
    if (pg >= p.max_blocks) return -1;
    if ((unsigned)row >= (unsigned)p.num_blocks) {
      bad = true;
      row = -1;
    }
    if (entry) p.block_table[(size_t)b * p.max_blocks + pg] = row;
    return row;
  };
  for (unsigned t0 = blockIdx.x * kTableThreads * U + tid * RUN; t0 < end; t0 += step) {
    if constexpr (RUN == 1) {
      int b[U], pos[U], row[U];
      unsigned t[U];
#pragma unroll
      for (int k = 0; k < U; ++k) {
        t[k] = t0 + k * kTableThreads;
        b[k] = 0;
      }
      // the last request that starts at or before the token (those without tokens are passed over)
      for (int d = top; d > 0; d >>= 1)
#pragma unroll
        for (int k = 0; k < U; ++k)
          if (b[k] + d < p.B && (unsigned)s_start[b[k] + d] <= t[k]) b[k] += d;
      const int32_t *src[U];
#pragma unroll
      for (int k = 0; k < U; ++k) {
        pos[k] = -1;
        src[k] = nullptr;
        if (t[k] >= tokens) continue;
        pos[k] = s_len[b[k]] + ((int)t[k] - s_start[b[k]]);
        src[k] = page_source(b[k], page_of(p, pos[k]), pages_had(b[k]));
      }
#pragma unroll
      for (int k = 0; k < U; ++k) row[k] = src[k] ? *src[k] : -1;
#pragma unroll
      for (int k = 0; k < U; ++k) {
        int slot = -1;
        if (pos[k] >= 0) {
          const int pg = page_of(p, pos[k]), off = pos[k] - pg * p.block_size;
          row[k] = checked(row[k], b[k], pg, off == 0 && pg >= pages_had(b[k]));
          if (row[k] >= 0) slot = row[k] * p.block_size + off;
        }
        if (t[k] < end) {
          p.slots[t[k]] = slot;
          p.positions[t[k]] = pos[k];
        }
      }
    } else {
      int slot[U], pos[U];
      int b = 0, have = 0, pg = 0, off = 0, row = -1, last = -1;
      unsigned stop = 0;  // the first token of the next request
#pragma unroll
      for (int k = 0; k < U; ++k) {
        slot[k] = pos[k] = -1;
        const unsigned t = t0 + k;
        if (t >= tokens) continue;
        bool look = false;  // the page's id has to be read
        if (t >= stop) {
          for (int d = top; d > 0; d >>= 1)
            if (b + d < p.B && (unsigned)s_start[b + d] <= t) b += d;
          stop = (unsigned)s_start[b + 1];
          const int len = s_len[b];
          have = pages_had(b);
          pos[k] = len + ((int)t - s_start[b]);
          pg = page_of(p, pos[k]);
          off = pos[k] - pg * p.block_size;
          look = true;
        } else {
          pos[k] = last + 1;
          if (++off == p.block_size) {
            off = 0;
            ++pg;
            look = true;
          }
        }
        last = pos[k];
        if (look) {
          const int32_t *src = page_source(b, pg, have);
          row = checked(src ? *src : -1, b, pg, off == 0 && pg >= have);
        }
        if (row >= 0) slot[k] = row * p.block_size + off;
      }
      if (t0 + U <= end) {
        *reinterpret_cast<int4 *>(p.slots + t0) = make_int4(slot[0], slot[1], slot[2], slot[3]);
        *reinterpret_cast<int4 *>(p.positions + t0) = make_int4(pos[0], pos[1], pos[2], pos[3]);
      } else {
#pragma unroll
        for (int k = 0; k < U; ++k)
          if (t0 + k < end) {
            p.slots[t0 + k] = slot[k];
            p.positions[t0 + k] = pos[k];
          }
      }
    }
  }
  if (bad) set_status(p.status, SV_DEV_BAD_BLOCK);
  if (report) {
    for (int b = tid; b <= p.B; b += kTableThreads) p.token_start[b] = s_start[b];
    if (tid == 0) {
      p.out_free_head[0] = (int)min(head + pages, (long long)INT32_MAX);
      if (total > p.T) set_status(p.status, SV_DEV_BAD_PREFIX);
      if (head < 0 || (pages > 0 && head + pages > p.num_free)) set_status(p.status, SV_DEV_BAD_BLOCK);
    }
  }
  if (total > p.T) pages_past_the_map<HELD>(p, table_smem, head, pages);
}

}  // namespace

cudaError_t launch_block_tables(TableParams p, int num_sms, cudaStream_t s) {
  const long long cap = (long long)p.max_blocks * p.block_size;
  p.cap = (int)(cap < INT32_MAX ? cap : INT32_MAX);
  p.div_shift = 0;
  while ((1ll << p.div_shift) < p.block_size) ++p.div_shift;
  p.div_mul = (unsigned)(((1ull << 32) * ((1ull << p.div_shift) - p.block_size)) / p.block_size + 1);
  // Many tokens per request: four neighbouring ones per thread.  Else CTAs of 256 threads with two
  // tokens each, so that few tokens go over many SMs, while the sums over the batch that every CTA
  // makes are short; beyond 2048 requests 1024 threads (256 requests of 5 tokens 3.7 us against 5.2,
  // 2048 of 5 5.6 against 6.6; 4096 of 32 9.1 against 7.4; device time).
  struct Form {
    void (*kernel)(TableParams);
    int threads, tokens;  // tokens that a CTA takes in a step
  };
  static const Form forms[6] = {{block_tables_kernel<4, 512, false>, 512, 2048},
                                {block_tables_kernel<1, 256, false>, 256, 512},
                                {block_tables_kernel<1, 1024, false>, 1024, 2048},
                                {block_tables_kernel<4, 512, true>, 512, 2048},
                                {block_tables_kernel<1, 256, true>, 256, 512},
                                {block_tables_kernel<1, 1024, true>, 1024, 2048}};
  const int form = (p.T / p.B >= 256 ? 0 : (p.B <= 2048 ? 1 : 2)) + (p.held ? 3 : 0);
  const Form &f = forms[form];
  const size_t smem = (size_t)((p.held ? 4 : 3) * p.B + 1) * sizeof(int);
  static std::atomic<bool> attr_set[6][64];
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev < 0 || dev >= 64 || !attr_set[form][dev].load()) {
    const cudaError_t e = cudaFuncSetAttribute(f.kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               (int)((4 * SV_MAX_TABLE_BATCH + 1) * sizeof(int)));
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < 64) attr_set[form][dev].store(true);
  }
  // (and, should there be more new tokens than places, CTAs for the table's entries: at most 64 a thread
  // as long as two CTAs per SM are enough for that)
  long long ctas = std::max(((long long)p.T + f.tokens - 1) / f.tokens, (long long)p.B * p.max_blocks / (64 * f.threads));
  ctas = ctas < 1 ? 1 : (ctas > 2ll * num_sms ? 2ll * num_sms : ctas);
  return launch_close(f.kernel, dim3((unsigned)ctas), f.threads, smem, s, p);
}

}  // namespace sv
