// Attention of many query rows over keys that they all see, on the 5th-generation tensor cores (tcgen05,
// TMEM, TMA; sm_103a, bf16): the shared part of sv_shared_attention and the listed pages of
// sv_sparse_attention where one list serves many rows.
//
// Sequences that share a prefix have, at each of its keys, K and V in common, so that their query rows
// (tokens x group heads) stack up to one matrix per KV head: S = Q K^T and O = P V over the prefix are
// matrix products like a prompt's, and K and V are read once per 256 rows instead of once per sequence.
// What differs by row (a sequence's own keys, the tree's mask) is not here: this kernel leaves each
// row's unnormalised output, maximum and sum over the keys that it has worked on, and the kernel of
// stacked_keys.cuh, which takes the own keys and the tree, joins them by softmax's rule
//   m = max m_i,  l = sum 2^(m_i - m) l_i,  o = sum 2^(m_i - m) o_i / l.
//
// Work: a unit is a KV head and up to 256 rows of a group (two MMA tiles A and B of 128), against the
// group's keys in tiles of 128.  The flattened (unit, key tile) space of W items is split evenly over min(W,
// SMs) persistent CTAs, so that each has at least one item; a unit that a CTA boundary cuts leaves one piece
// per CTA.  Piece number = unit + CTA, which is unique, since one of the two grows from piece to piece.
//
// Per CTA: a copying warp (TMA: Q per piece, K and V tiles through a ring), an issuing warp (one elected
// thread), and two groups of four softmax warps, one thread per row, a group per MMA tile.  P goes back to TMEM
// over the S it came from.  The issue order is S_A S_B | P_A V, S_A', P_B V, S_B' | ...: one tile's softmax
// runs beside the other's products.  MMAs of one thread run in the order of their issue, so that S'
// may be issued over P as soon as P V has been, without waiting for it.
//
// Bound by the CTA's chain of products and softmax: 32 sequences with 64 nodes each behind one prompt of 4099 keys,
// 32:32 heads of 128, 94 us, 1.45 PFLOP/s, the tensor pipe 68 % active, the unit of the exponents a third (pages of 16
// instead of a contiguous cache: 7 % more; over lists the pipe is 51 % active, for reasons not found).
// (With half of the MMAs left out 84.5 us, with the exponents left out no change.)  What was tried: 16 softmax warps, half
// a row each, 102 us against 96; weights of the first half against the maximum of the tile before 100.6
// against 95.6; four stages of the ring and page ids tile by tile, 256 requests in four groups, 104 against 98; tiles
// prefetched to the L2 115 against 97.
#include <atomic>
#include <cfloat>

#include "sv_common.cuh"
#include "sv_internal.h"
#include "tc_primitives.cuh"

namespace sv {

namespace {

using namespace tc;

constexpr int kRows = 128;               // rows of an MMA tile
constexpr int kKeys = 128;               // keys of a tile
constexpr float kStackRescale = 8.f;     // log2 units by which a row's maximum may lag behind
constexpr float kStackNone = -3e38f;     // a row's maximum before its first key
constexpr int kStackThreads = 384;       // two softmax groups; copies, issue and two warps without work
constexpr unsigned long long kAllKeys = 0x1010101010101010ull;  // 16 keys in each of 8 chunks

template <int D>
struct StackLayout {
  static constexpr int KB = D / 64;                 // 64-column blocks
  static constexpr int Q_TILE = kRows * D * 2;      // rows of an MMA tile
  static constexpr int KV_BYTES = kKeys * D * 2;    // K or V of a key tile
  static constexpr int ST = D == 128 ? 5 : 10;      // stages of the ring, K and V in turn
  static constexpr int OFF_RING = 2 * Q_TILE;
  static constexpr int OFF_BAR = OFF_RING + ST * KV_BYTES;
  // full[ST], empty[ST], q_full, q_empty, s_full[2], p_half[2], p_full[2], o_full[2], drain
  static constexpr int NBAR = 2 * ST + 11;
  static constexpr int OFF_KEYS = OFF_BAR + NBAR * 8;   // [8] keys of each chunk of a tile
  static constexpr int OFF_MISC = OFF_KEYS + 8 * 8;     // TMEM address, abort
  static constexpr int OFF_WORK = OFF_MISC + 16;        // [groups + 1] first work item of a group
  static constexpr int OFF_UNIT = OFF_WORK + (SV_MAX_SHARED_GROUPS + 1) * 8;  // [groups] its first unit
  static constexpr int SMEM = OFF_UNIT + SV_MAX_SHARED_GROUPS * 4;
  static_assert(SMEM <= 227 * 1024, "shared memory");
};

// A piece: key tiles [t0, t1) of a unit.
struct StackPiece {
  int head, first, token, tokens, t0, t1, slot, keys, list;
};

// A group of sequences: what its rows are and how many keys they share (a multiple of 16).
struct StackGroup {
  int start, members, keys, tiles;
};
__device__ __forceinline__ StackGroup stack_group(const StackParams &p, int g) {
  StackGroup a;
  a.start = p.group_start[g];
  a.members = p.group_start[g + 1] - a.start;
  a.keys = min(max(p.shared_len[g], 0), p.cap) & ~15;
  a.tiles = a.members > 0 ? (a.keys + kKeys - 1) / kKeys : 0;
  return a;
}

struct StackTables {
  const long long *work;
  const int *unit;
};

// Walks a CTA's share [w, end) of the work, piece by piece.
struct StackWalk {
  long long w, end;
  int g;
};
template <bool LIST>
__device__ __forceinline__ bool next_piece(StackWalk &it, const StackParams &p, const StackTables &t, StackPiece &pc) {
  if (it.w >= it.end) return false;
  int kt;
  if constexpr (LIST) {
    kt = p.list_tiles;
    const long long u = it.w / kt;
    pc.t0 = (int)(it.w - u * kt);
    const int tile = (int)(u % p.row_tiles), bh = (int)(u / p.row_tiles);
    pc.list = bh;
    pc.head = bh % p.Hkv;
    pc.first = bh / p.Hkv;
    pc.token = pc.first * p.N + tile * 2 * p.tile_tokens;
    pc.tokens = min(2 * p.tile_tokens, p.N - tile * 2 * p.tile_tokens);
    pc.keys = 0;
    pc.slot = (int)u + (int)blockIdx.x;
  } else {
    while (it.w >= t.work[it.g + 1]) ++it.g;
    const StackGroup g = stack_group(p, it.g);
    kt = g.tiles;
    const int u = (int)((it.w - t.work[it.g]) / kt);
    pc.t0 = (int)(it.w - t.work[it.g] - (long long)u * kt);
    const int total = g.members * p.N, per = (total + 2 * p.tile_tokens - 1) / (2 * p.tile_tokens);
    const int tile = u % per;
    pc.head = u / per;
    pc.first = g.start;
    pc.token = pc.first * p.N + tile * 2 * p.tile_tokens;
    pc.tokens = min(2 * p.tile_tokens, total - tile * 2 * p.tile_tokens);
    pc.keys = g.keys;
    pc.list = 0;
    pc.slot = t.unit[it.g] + u + (int)blockIdx.x;
  }
  pc.t1 = (int)min((long long)kt, pc.t0 + (it.end - it.w));
  it.w += pc.t1 - pc.t0;
  return true;
}

// A lane's chunk of 16 keys of a key tile (lanes 0 to 7).
struct ChunkRows {
  int row;    // of the cache, -1: none
  int count;  // keys
};

__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{.reg .b64 ra, rb, rc, rd;\n mov.b64 ra, {%2, %3};\n mov.b64 rb, {%4, %5};\n mov.b64 rc, {%6, %7};\n"
      " fma.rn.f32x2 rd, ra, rb, rc;\n mov.b64 {%0, %1}, rd;}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}

// Wait for the phase of the given parity; false if it ran past the limit (then *abort is raised) or *abort
// was raised.  (Inline: with a function call in it ptxas finds no registers for the split below.)
__device__ __forceinline__ bool stack_wait(uint64_t *bar, uint32_t parity, volatile int *abort, unsigned long long limit) {
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

// LIST: listed pages; GROUPED: pages that come with both 64-column halves in one copy, as groups of 8 rows.
template <int D, bool LIST, bool GROUPED>
__global__ void __launch_bounds__(kStackThreads, 1) stacked_attn_kernel(const __grid_constant__ StackParams p) {
  using Lay = StackLayout<D>;
  constexpr int ST = Lay::ST, KB = Lay::KB;
  extern __shared__ __align__(1024) uint8_t stack_smem[];
  uint8_t *sm = stack_smem;
  uint64_t *full = reinterpret_cast<uint64_t *>(sm + Lay::OFF_BAR), *empty = full + ST;
  uint64_t *q_full = empty + ST, *q_empty = q_full + 1, *s_full = q_empty + 1, *p_half = s_full + 2, *p_full = p_half + 2,
           *o_full = p_full + 2, *drain = o_full + 2;
  volatile unsigned long long *s_keys = reinterpret_cast<volatile unsigned long long *>(sm + Lay::OFF_KEYS);
  uint32_t *s_tmem = reinterpret_cast<uint32_t *>(sm + Lay::OFF_MISC);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(s_tmem + 1);
  long long *s_work = reinterpret_cast<long long *>(sm + Lay::OFF_WORK);
  int *s_unit = reinterpret_cast<int *>(sm + Lay::OFF_UNIT);
  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xFFFFFFFFu, tid >> 5, 0);
  const unsigned long long limit = p.wait_ns;

  const bool layout_ok = (smem_u32(sm) & 1023u) == 0;  // 128-byte-swizzled tiles
  if (tid == 0) {
    for (int i = 0; i < ST; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    mbar_init(q_full, 1);
    mbar_init(q_empty, 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&p_half[i], 4);
      mbar_init(&p_full[i], 4);
      mbar_init(&o_full[i], 1);
    }
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 9) {
    tmem_alloc(s_tmem, 512);
    tmem_relinquish();
  }
  wait_previous();
  // The kernel behind this one may be set up from here on: it reads what was there before this one, and
  // waits for this one before it reads the pieces.
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  // ---- the work: units and key tiles of each group
  long long total = p.list_work;
  if constexpr (!LIST) {
    int bad = 0;
    for (int g = tid; g < p.groups; g += kStackThreads) {
      const int a = p.group_start[g], b = p.group_start[g + 1], len = p.shared_len[g];
      bad |= a < 0 || b < a || b > p.B;
      if (blockIdx.x == 0 && (len < 0 || len > p.cap)) set_status(p.status, SV_DEV_BAD_PREFIX);
    }
    bad = __syncthreads_or(bad);
    if (bad && tid == 0 && blockIdx.x == 0) set_status(p.status, SV_DEV_BAD_GROUP);
    if (warp == 0) {
      long long work = 0;
      int units = 0;
      for (int g0 = 0; g0 < p.groups && !bad; g0 += 32) {
        const int g = g0 + lane;
        int n = 0, tiles = 0;
        if (g < p.groups) {
          const StackGroup a = stack_group(p, g);
          tiles = a.tiles;
          if (tiles > 0) n = (a.members * p.N + 2 * p.tile_tokens - 1) / (2 * p.tile_tokens) * p.Hkv;
        }
        long long x = (long long)n * tiles;
        const long long mine_x = x;
        const int mine_n = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const long long y = __shfl_up_sync(0xFFFFFFFFu, x, o);
          const int k = __shfl_up_sync(0xFFFFFFFFu, n, o);
          if (lane >= o) x += y, n += k;
        }
        if (g < p.groups) {
          s_work[g] = work + x - mine_x;
          s_unit[g] = units + n - mine_n;
          // for the kernel that joins the pieces
          if (blockIdx.x == 0) {
            p.header[1 + 2 * g] = work + x - mine_x;
            p.header[2 + 2 * g] = (long long)tiles << 32 | (unsigned)(units + n - mine_n);
          }
        }
        work += __shfl_sync(0xFFFFFFFFu, x, 31);
        units += __shfl_sync(0xFFFFFFFFu, n, 31);
      }
      if (lane == 0) s_work[p.groups] = work;
      if (blockIdx.x == 0 && lane == 0) p.header[0] = work;
    }
    __syncthreads();
    total = s_work[p.groups];
  } else {
    __syncthreads();
  }
  tc_fence_after();
  const uint32_t tmem = *s_tmem;
  const StackTables tables{s_work, s_unit};
  // every CTA that takes part has work, so that a unit's pieces are those of neighbouring CTAs
  const long long ctas = min((long long)gridDim.x, total);
  StackWalk walk{0, 0, 0};
  if (blockIdx.x < ctas && layout_ok) walk = {total * blockIdx.x / ctas, total * (blockIdx.x + 1) / ctas, 0};
  uint8_t *ring = sm + Lay::OFF_RING;
  int copied = 0, q_copied = 0;  // (the copying warp) stages filled, pieces begun

  if (warp >= 8) {
    // 168 registers per thread at the launch, 64512 in all: 128 threads keep 88, 256 take 208
    asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
    if (warp == 8) {
      // ---------------------------------------------------------------- copies
      const uint64_t policy = l2_policy_evict_normal();
      int tiles = 0;  // key tiles
      // this lane's chunk of key tile t (lanes 8 j to 8 j + 7: tile j of four, whose ids are read together)
      auto locate = [&](const StackPiece &pc, int t) -> ChunkRows {
        ChunkRows c{-1, 0};
        if (t >= pc.t1) return c;
        const int at = t * kKeys + 16 * (lane & 7);
        int page = 0, off, pos, count = 16;
        if constexpr (LIST) {
          const int k = at / p.page_size;
          if (k >= p.list_len) return c;
          page = p.pages[(size_t)pc.list * p.list_len + k];
          off = at - k * p.page_size;
          const long long far = (long long)page * p.page_size + off;
          const int L = min(max(p.prefix_len[pc.first], 0), p.cap);
          if (page < 0 || far >= L) return c;
          pos = (int)far;
          count = min(16, L - pos);
        } else {
          if (at >= pc.keys) return c;
          pos = at;
          if (p.block_table) page = pos / p.block_size;
          off = pos - page * p.block_size;
        }
        if (!p.block_table) return ChunkRows{pc.first * p.Lmax + pos, count};
        const int blk = p.block_table[(size_t)pc.first * p.max_blocks + page];
        if (blk < 0 || blk >= p.num_blocks) {
          set_status(p.status, SV_DEV_BAD_BLOCK);
          return c;
        }
        return ChunkRows{blk * p.block_size + off, count};
      };
      const int per_box = p.box_rows / 16;  // chunks of a box
      // the next stage: K or V of the tile whose rows the lanes hold
      auto load = [&](const StackPiece &pc, const ChunkRows &c, int j, bool is_v) -> bool {
        const int st = copied % ST;
        int ok = 1;
        if (copied >= ST && lane == 0) ok = stack_wait(&empty[st], (copied / ST - 1) & 1, abort_flag, limit);
        if (!__shfl_sync(0xFFFFFFFFu, ok, 0)) return false;
        const bool mine = lane >> 3 == j, box = mine && (lane & 7) % per_box == 0 && c.row >= 0;
        const unsigned boxes = __popc(__ballot_sync(0xFFFFFFFFu, box));
        if (!is_v) {
          const unsigned lo = __reduce_or_sync(0xFFFFFFFFu, mine && !(lane & 4) ? (unsigned)c.count << (8 * (lane & 3)) : 0u);
          const unsigned hi = __reduce_or_sync(0xFFFFFFFFu, mine && (lane & 4) ? (unsigned)c.count << (8 * (lane & 3)) : 0u);
          if (lane == 0) s_keys[tiles & 7] = (unsigned long long)hi << 32 | lo;
        }
        if (lane == 0) mbar_expect_tx(&full[st], boxes * (unsigned)p.box_rows * D * 2u);
        __syncwarp();
        uint8_t *dst = ring + st * Lay::KV_BYTES;
        const CUtensorMap *map = is_v ? &p.tm_v : &p.tm_k;
        if (box) {
          if (GROUPED) {
            tma_load_5d_hint(dst + (lane & 7) * 16 * (D * 2), map, 0, 0, 0, c.row >> 3, pc.head, &full[st], policy);
          } else {
#pragma unroll
            for (int k = 0; k < KB; ++k)
              tma_load_3d_hint(dst + k * (kKeys * 128) + (lane & 7) * 16 * 128, map, 64 * k, pc.head, c.row, &full[st], policy);
          }
        }
        ++copied;
        return true;
      };
      StackPiece pc;
      bool ok = true;
      while (ok && next_piece<LIST>(walk, p, tables, pc)) {
        ChunkRows rows{-1, 0};
        for (int t = pc.t0; ok && t < pc.t1; ++t) {
          const int j = (t - pc.t0) & 3;
          if (j == 0) rows = locate(pc, t + (lane >> 3));
          ok = load(pc, rows, j, false);
          if (ok && t == pc.t0) {
            int free = 1;
            if (q_copied > 0 && lane == 0) free = stack_wait(q_empty, (q_copied - 1) & 1, abort_flag, limit);
            ok = __shfl_sync(0xFFFFFFFFu, free, 0);
            if (ok && lane == 0) {
              const int n = pc.tokens > p.tile_tokens ? 2 : 1;
              mbar_expect_tx(q_full, (unsigned)(n * p.tile_tokens * p.G) * D * 2u);
              for (int i = 0; i < n; ++i)
                for (int k = 0; k < KB; ++k)
                  tma_load_3d(sm + i * Lay::Q_TILE + k * (kRows * 128), &p.tm_q, 64 * k, pc.head * p.G,
                              pc.token + i * p.tile_tokens, q_full);
            }
            if (ok) ++q_copied;
          }
          if (ok) ok = load(pc, rows, j, true);
          ++tiles;
        }
      }
    } else if (warp == 9) {
      // ----------------------------------------------------------------- issue
      // The whole warp walks and waits, so that what the elected thread issues is in uniform registers
      // (one thread alone in this loop: 147 cycles per MMA instead of 75).
      constexpr uint32_t id_s = idesc_bf16(kRows, kKeys, 0, 0), id_o = idesc_bf16(kRows, D, 0, 1);
      constexpr uint32_t kBlock = GROUPED ? 1024 : kKeys * 128, kStep8 = GROUPED ? KB * 1024 : 1024;
      const uint64_t dq = sdesc_sw128(smem_u32(sm), 16, 1024);
      const uint64_t dk = sdesc_sw128(smem_u32(ring), 16, kStep8), dv = sdesc_sw128(smem_u32(ring), kBlock, kStep8);
      const uint32_t tm = __shfl_sync(0xFFFFFFFFu, tmem, 0);
      int pieces = 0, na = 0, nb = 0;  // pieces, key tiles of A and of B
      int st = 0, par = 0;             // the next stage and its parity
      auto uniform = [](int v) { return __shfl_sync(0xFFFFFFFFu, v, 0); };  // (the same in every lane, and known to be)
      auto arrived = [&](uint64_t *bar, int parity) -> bool {
        return __all_sync(0xFFFFFFFFu, stack_wait(bar, parity, abort_flag, limit));
      };
      auto next_stage = [&]() {
        if (++st == ST) st = 0, par ^= 1;
      };
      auto scores = [&](int x, int at) {
        const uint64_t a = dq + (uint64_t)(x * Lay::Q_TILE >> 4), b = dk + (uint64_t)(at * (Lay::KV_BYTES >> 4));
        if (elect_one()) {
#pragma unroll
          for (int k = 0; k < D / 16; ++k)
            umma_bf16(tm + x * kKeys, a + (uint64_t)(((k >> 2) * (kRows * 128) + (k & 3) * 32) >> 4),
                      b + (uint64_t)(((k >> 2) * kBlock + (k & 3) * 32) >> 4), id_s, k > 0);
          umma_commit(&s_full[x]);
        }
        __syncwarp();
      };
      auto outputs = [&](int x, int at, bool first, int n) -> bool {
        const uint64_t v = dv + (uint64_t)(at * (Lay::KV_BYTES >> 4));
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if (!arrived(h ? &p_full[x] : &p_half[x], n & 1)) return false;
          tc_fence_after();
          if (elect_one()) {
#pragma unroll
            for (int k = 4 * h; k < 4 * h + 4; ++k)
              umma_bf16_ts(tm + 256 + x * D, tm + x * kKeys + k * 8, v + (uint64_t)(k * 2 * kStep8 >> 4), id_o,
                           (!first || k > 0) ? 1u : 0u);
          }
          __syncwarp();
        }
        return true;
      };
      auto commit = [&](uint64_t *bar) {
        if (elect_one()) umma_commit(bar);
        __syncwarp();
      };
      StackPiece pc;
      bool ok = true;
      while (ok && uniform(next_piece<LIST>(walk, p, tables, pc))) {
        const bool two = uniform(pc.tokens > p.tile_tokens);
        const int n = uniform(pc.t1 - pc.t0);
        ok = arrived(q_full, pieces & 1) && arrived(&full[st], par);
        if (!ok) break;
        tc_fence_after();
        scores(0, st);
        if (two) scores(1, st);
        commit(&empty[st]);
        if (n == 1) commit(q_empty);
        next_stage();
        for (int i = 0; i < n; ++i) {
          const int sv = st, pv = par;
          next_stage();
          const bool more = i + 1 < n;
          ok = arrived(&full[sv], pv) && (!more || arrived(&full[st], par)) &&
               outputs(0, sv, i == 0, na);
          if (!ok) break;
          ++na;
          if (more) scores(0, st);
          else commit(&o_full[0]);
          if (two) {
            ok = outputs(1, sv, i == 0, nb);
            if (!ok) break;
            ++nb;
          }
          commit(&empty[sv]);
          if (more) {
            if (two) scores(1, st);
            commit(&empty[st]);
            if (i + 2 == n) commit(q_empty);
            next_stage();
          } else if (two) {
            commit(&o_full[1]);
          }
        }
        ++pieces;
      }
      // every MMA has completed before TMEM is given up
      commit(drain);
      const unsigned long long t0 = global_ns();
      while (!mbar_try_wait(drain, 0) && global_ns() - t0 < kWaitLimitNs) {
      }
    }
  } else {
    // ----------------------------------------------------------------- softmax
    asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
    const int x = warp >> 2, wq = warp & 3, row = wq * 32 + lane;
    const uint32_t lanes = (uint32_t)(wq * 32) << 16;
    const uint32_t ts = tmem + lanes + x * kKeys, to = tmem + lanes + 256 + x * D;
    const float sc = p.scale_log2;
    // (a warp goes on or leaves as a whole: behind each wait are operations that all of its lanes take part in)
    auto arrived = [&](uint64_t *bar, int parity) -> bool {
      return __all_sync(0xFFFFFFFFu, stack_wait(bar, parity, abort_flag, limit));
    };
    int r = 0, tiles = 0, n = 0, done = 0;  // stages, key tiles of the CTA, of this MMA tile, pieces of this MMA tile
    StackPiece pc;
    bool ok = true;
    while (ok && next_piece<LIST>(walk, p, tables, pc)) {
      const int rows = min(p.tile_tokens, pc.tokens - x * p.tile_tokens) * p.G;  // of this MMA tile
      if (rows <= 0) {
        r += 2 * (pc.t1 - pc.t0);
        tiles += pc.t1 - pc.t0;
        continue;
      }
      const bool idle = wq * 32 >= rows;  // padding: the barriers only
      // (the other rows of a tile hold another sequence's queries, or what was in shared memory before: they move no
      // maximum of the warp's)
      const bool real = row < rows;
      float m = kStackNone, l = 0.f;
      for (int t = pc.t0; t < pc.t1; ++t, ++tiles, ++n, r += 2) {
        if (!arrived(&s_full[x], n & 1)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const unsigned long long keys = s_keys[tiles & 7];
        if (keys != kAllKeys && x == 0) {
          // V rows that are no keys may hold anything: zero, so that 0 * V stays 0
          const int sv = (r + 1) % ST;
          if (!arrived(&full[sv], ((r + 1) / ST) & 1)) {
            ok = false;
            break;
          }
          uint8_t *v = ring + sv * Lay::KV_BYTES;
          for (int i = tid; i < kKeys * (D / 8); i += 128) {
            const int k = i / (D / 8), c = i % (D / 8);
            if ((k & 15) < (int)(keys >> (8 * (k >> 4)) & 31)) continue;
            uint8_t *at = GROUPED ? v + (k >> 3) * (KB * 1024) + (c >> 3) * 1024 + (k & 7) * 128 + (c & 7) * 16
                                    : v + (c >> 3) * (kKeys * 128) + k * 128 + (c & 7) * 16;
            // (whole rows are zeroed, so that the swizzle of their 16-byte chunks does not matter)
            *reinterpret_cast<uint4 *>(at) = make_uint4(0, 0, 0, 0);
          }
          fence_proxy_async_smem();
        }
        if (!idle) {
          float s[4][32];
#pragma unroll
          for (int c = 0; c < 4; ++c) tmem_ld32(ts + 32 * c, s[c]);
          tmem_wait_ld();
          if (keys != kAllKeys) {
#pragma unroll
            for (int c = 0; c < 8; ++c) {
              const int count = (int)(keys >> (8 * c) & 31);
#pragma unroll
              for (int i = 0; i < 16; ++i)
                if (i >= count) s[c >> 1][16 * (c & 1) + i] = -INFINITY;
            }
          }
          float top[4];
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            top[c] = fmaxf(s[c][0], s[c][1]);
#pragma unroll
            for (int i = 2; i < 32; i += 2) top[c] = fmax3(top[c], s[c][i], s[c][i + 1]);
          }
          const float best = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])) * sc;
          const bool moves = real && best > m + kStackRescale;
          if (__any_sync(0xFFFFFFFFu, moves)) {
            const float to_m = fmaxf(best, m), w = ex2_approx(m - to_m);
            m = to_m;
            l *= w;
            if (t > pc.t0) {  // (S of this tile is there, so P V of the tile before is done)
#pragma unroll 1
              for (int c = 0; c < D; c += 16) {
                float o[16];
                tmem_ld16(to + c, o);
                tmem_wait_ld();
#pragma unroll
                for (int i = 0; i < 16; ++i) o[i] *= w;
                tmem_st16(to + c, o);
              }
            }
          }
          const float2 sc2 = make_float2(sc, sc), m2 = make_float2(-m, -m);
          float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            float w[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              float2 e = fma2(make_float2(s[c][2 * i], s[c][2 * i + 1]), sc2, m2);
              e.x = ex2_approx(e.x);
              e.y = ex2_approx(e.y);
              sum[i & 1] = add2(sum[i & 1], e);
              // (rounded to bf16 for the product with V, at most 2^-8 of each; the sum is of the unrounded)
              w[i] = __uint_as_float(pack_bf16x2(e.x, e.y));
            }
            tmem_st16(ts + 16 * c, w);
            if (c == 1) {
              tmem_wait_st();
              tc_fence_before();
              __syncwarp();
              if (lane == 0) mbar_arrive(&p_half[x]);
            }
          }
          const float2 both = add2(sum[0], sum[1]);
          l += both.x + both.y;
          tmem_wait_st();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&p_full[x]);
        } else {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(&p_half[x]);
            mbar_arrive(&p_full[x]);
          }
        }
      }
      if (!ok) break;
      if (!arrived(&o_full[x], done & 1)) break;
      ++done;
      tc_fence_after();
      if (!idle) {
        const int in = x * kRows + row;
        if (real) p.part_ml[(size_t)pc.slot * kStackRows + in] = make_float2(m, l);
        // by 16 bytes of all rows, so that a warp's stores are 512 bytes side by side (row by row: 2 us more
        // per piece)
        float4 *to_o = reinterpret_cast<float4 *>(p.part_o) + (size_t)pc.slot * (D / 4) * kStackRows + in;
#pragma unroll 1
        for (int c = 0; c < D; c += 32) {
          float o[32];
          tmem_ld32(to + c, o);
          tmem_wait_ld();
          if (real) {
#pragma unroll
            for (int i = 0; i < 32; i += 4) to_o[(size_t)((c + i) / 4) * kStackRows] = make_float4(o[i], o[i + 1], o[i + 2], o[i + 3]);
          }
        }
        tc_fence_before();  // (the next piece's first P V comes behind this warp's next arrival)
      }
    }
  }
  __syncthreads();
  if (warp == 8 && lane == 0 && *abort_flag) {
    // a wait gave up: let the copies in flight land before the CTA's shared memory is given up
    const unsigned long long t0 = global_ns();
    for (int i = max(0, copied - ST); i < copied; ++i)
      while (!mbar_try_wait(&full[i % ST], (i / ST) & 1) && global_ns() - t0 < kWaitLimitNs) {
      }
    while (q_copied > 0 && !mbar_try_wait(q_full, (q_copied - 1) & 1) && global_ns() - t0 < kWaitLimitNs) {
    }
  }
  if (warp == 9) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
  if (tid == 0) {
    if (!layout_ok) set_status(p.status, SV_DEV_LAYOUT);
    else if (*abort_flag) set_status(p.status, SV_DEV_TIMEOUT);
  }
}

template <int D, bool LIST, bool GROUPED>
cudaError_t launch_stacked_typed(const StackParams &p, int grid, cudaStream_t s) {
  using Lay = StackLayout<D>;
  static std::atomic<bool> attr[64];
  int dev = 0;
  cudaGetDevice(&dev);
  auto kern = stacked_attn_kernel<D, LIST, GROUPED>;
  if (dev < 0 || dev >= 64 || !attr[dev].load()) {
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Lay::SMEM);
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < 64) attr[dev].store(true);
  }
  return launch_close(kern, dim3((unsigned)grid), kStackThreads, (size_t)Lay::SMEM, s, p);
}

}  // namespace

cudaError_t launch_stacked(const StackParams &p, int D, bool listed, int grid, cudaStream_t s) {
  if (D == 64) return listed ? launch_stacked_typed<64, true, false>(p, grid, s) : launch_stacked_typed<64, false, false>(p, grid, s);
  if (p.grouped) return listed ? launch_stacked_typed<128, true, true>(p, grid, s) : launch_stacked_typed<128, false, true>(p, grid, s);
  return listed ? launch_stacked_typed<128, true, false>(p, grid, s) : launch_stacked_typed<128, false, false>(p, grid, s);
}

}  // namespace sv
