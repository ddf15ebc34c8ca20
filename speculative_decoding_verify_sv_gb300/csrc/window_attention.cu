// Tree attention over a sliding window with sinks for units of few query rows (sm_103a, bf16).
//
// Node n of sequence b stands at P = L_b + depth(n); its keys are the prefix positions p with
// P - p < window or p < sinks, and the nodes of its root path by the same rule.  A unit is a
// sequence and KV head: its M = N * G query rows (tree nodes x group heads), in tiles of up to 64, against
//   the tree's N nodes, the sinks before the window, and [first, L_b),
// first = L_b - window + 1 being the earliest position that a row's window reaches (rounded
// down to 16 in a paged cache).  These keys are cut into groups of 16, none of which crosses a
// page.
//
// With few rows the work is a stream of K and V: what counts is that loads are always in
// flight and that units, which a window keeps short, begin and end without gaps.  So nothing
// in the main loop waits for another warp: each slice of a CTA (one warp; two with more than
// 32 rows in it, which then share a slice's rows) takes every KS-th group, has a ring of its own
// in shared memory, issues its own TMA copies (16 rows of a head per box, several groups ahead)
// and keeps its own running maximum, sum and output in registers.  Two CTAs share an SM, so one
// streams while the other starts or ends.
//
// The products are taken transposed, S^T = K Q^T and O^T = V^T P^T: keys and head
// dimensions fill the 16-row side of the matrix instruction and the query rows its 8-column
// side, so that 4 rows (one token, 4 group heads) cost one 8-column step and 20 rows cost
// three, where a 128-row tcgen05 tile would be padded to 128.  P^T goes from accumulator to
// operand layout by an 8x8 transpose in registers, rounded to bf16 (off by at most 2^-8 of each
// weight; the sum is of the unrounded ones); scores, weights, sums and outputs are fp32.
//
// Bound by HBM for many units of up to 48 rows: 256 ragged requests of 5 nodes, 32:8 heads of 128,
// window 1024 in pages of 16, 174 us, 6.2 TB/s, 91 % of the measured copy rate (the 128-row kernel
// 268 us); by the warps' chains of products and exponents for 64 rows (256 units, window 513: 23.8 us,
// of which 2 start, 16 loop, 2.5 merge; the matrix pipe is half busy); by latency for few units: one
// token of one request, window 1024, 5.5 us (the 128-row kernel 49).
//
// The slices merge in shared memory by weights 2^(m_slice - m), each taking some dimensions of all
// rows, as they stand in registers, and the results leave as 32-byte sectors by a transpose and an
// exchange between neighbours (5.3 thousand cycles -> 3.5 for 64 rows against rows of floats in shared
// memory).  Few long units: a cluster of up to 8 CTAs shares a unit's groups, without a workspace or
// a second launch; each CTA takes part of the unit's outputs, which the others write into its shared
// memory (reading them from there instead: 6.6 us against 5.5 for one token).
#include <algorithm>
#include <atomic>
#include <cfloat>
#include <cmath>
#include <type_traits>

#include "cluster.cuh"
#include "sv_common.cuh"
#include "sv_internal.h"
#include "tc_primitives.cuh"

namespace sv {

namespace {

using namespace tc;

constexpr int kWinThreads = 128;
constexpr int kWinGroup = 16;        // keys per group
constexpr float kWinRescale = 8.f;   // log2 units by which a row's maximum may run ahead
constexpr float kWinNone = -3e38f;   // a row's maximum before its first key

template <int D, int NT, int RG>
struct WinLayout {
  static constexpr int KS = 4 / RG;             // slices
  static constexpr int KB = D / 64;             // 64-column blocks of a row
  static constexpr int K_BYTES = kWinGroup * D * 2;
  static constexpr int G_BYTES = 2 * K_BYTES;   // a group's K and V
  // the slices' rings: what two CTAs per SM leave room for beside their query rows
  static constexpr int RING = (RG == 2 ? 80 : 96) * 1024;
  static constexpr int ST = RING / (KS * G_BYTES);  // stages of a slice's ring
  static constexpr int RB = 8 * NT * RG;        // query rows of a CTA
  static constexpr int DO = D / 16 / KS;        // 16-dimension tiles of the outputs that a slice merges
  static constexpr int UNITS = RG * D / 16 * NT;  // of the merge: 16 dimensions of 8 rows
  static constexpr int OFF_Q = RING;            // query rows [RB][D], 128-byte swizzle per 64 columns
  // in the ring's room, after the slices' parts: what the CTAs of a cluster hand over, outputs
  // [units], maxima and sums [8][RB]
  static constexpr int OFF_JOIN = (KS - 1) * UNITS * 512;
  static constexpr int JOIN = (UNITS + 8) * 512 + 2 * 8 * RB * 4;
  static constexpr int OFF_FULL = OFF_Q + RB * D * 2;
  static constexpr int OFF_EMPTY = OFF_FULL + KS * ST * 8;
  static constexpr int OFF_ANC = OFF_EMPTY + KS * ST * 8;
  static constexpr int OFF_M = OFF_ANC + RB * 8;        // [KS][RB]
  static constexpr int OFF_L = OFF_M + KS * RB * 4;     // [KS][RB]
  static constexpr int OFF_INV = OFF_L + KS * RB * 4;   // [RB] 1 / sum
  static constexpr int OFF_LO = OFF_INV + RB * 4;       // [RB]
  static constexpr int OFF_ROW = OFF_LO + RB * 4;       // [RB]
  static constexpr int OFF_PAR = OFF_ROW + RB * 4;      // [64]
  static constexpr int OFF_COPIED = OFF_PAR + kMaxNodes * 4;  // [KS][ST]
  static constexpr int OFF_ABORT = OFF_COPIED + KS * ST * 4;
  static constexpr int SMEM = OFF_ABORT + 16;
  static_assert(OFF_JOIN + JOIN <= RING, "the merge goes on in the ring's room");
  static_assert(SMEM <= 113 * 1024, "two CTAs per SM");
};

// Wait for the phase of the given parity; false if it ran past the limit (then *abort is raised) or
// *abort was raised.  A try suspends the thread for a time of the hardware's choice, or for a given one:
// behind the first try it is the limit, or a millisecond, so that short limits count (those up to a
// millisecond with the first try) and an abort is seen soon.  (A time given to the first try too costs 2 %.)
__device__ __forceinline__ bool try_wait_for(uint64_t *bar, uint32_t parity, uint32_t ns) {
  uint32_t ok;
  asm volatile("{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n selp.u32 %0, 1, 0, p;\n}\n"
               : "=r"(ok)
               : "r"(smem_u32(bar)), "r"(parity), "r"(ns)
               : "memory");
  return ok != 0;
}
constexpr unsigned kWinTryNs = 1000000;
__device__ __noinline__ bool limited_wait_slow(uint64_t *bar, uint32_t parity, volatile int *abort, uint32_t ns,
                                               unsigned long long limit_ns) {
  const unsigned long long t0 = global_ns() - ns;  // (the first try)
  while (!*abort && global_ns() - t0 < limit_ns)
    if (try_wait_for(bar, parity, ns)) return true;
  *abort = 1;
  return false;
}
__device__ __forceinline__ bool limited_wait(uint64_t *bar, uint32_t parity, volatile int *abort, const WinParams &p) {
  return mbar_try_wait(bar, parity) || limited_wait_slow(bar, parity, abort, p.try_ns, p.wait_ns);
}
// True in one lane of a converged warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t one;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xFFFFFFFF;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(one));
  return one != 0;
}
// Transpose of an 8x8 matrix of 16-bit elements held in fragment layout by a warp.
__device__ __forceinline__ uint32_t transpose_8x8(uint32_t a) {
  uint32_t d;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}

// ldmatrix from a shared-memory address.
__device__ __forceinline__ void ldsm_x4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];\n"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}
__device__ __forceinline__ void ldsm_x4_trans(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];\n"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}

// A product that starts a sum.
__device__ __forceinline__ void mma_first(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};\n"
               : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
               : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}

template <int D, int NT, int RG>
__global__ void __launch_bounds__(kWinThreads, 2) window_attn_kernel(const __grid_constant__ WinParams p) {
  using Lay = WinLayout<D, NT, RG>;
  constexpr int KS = Lay::KS, KB = Lay::KB, ST = Lay::ST, RB = Lay::RB, DT = D / 16;
  extern __shared__ __align__(1024) uint8_t win_smem[];
  uint8_t *sm = win_smem;
  uint64_t *s_anc = reinterpret_cast<uint64_t *>(sm + Lay::OFF_ANC);
  float *s_m = reinterpret_cast<float *>(sm + Lay::OFF_M), *s_l = reinterpret_cast<float *>(sm + Lay::OFF_L);
  float *s_inv = reinterpret_cast<float *>(sm + Lay::OFF_INV);
  int *s_lo = reinterpret_cast<int *>(sm + Lay::OFF_LO), *s_par = reinterpret_cast<int *>(sm + Lay::OFF_PAR);
  int *s_row = reinterpret_cast<int *>(sm + Lay::OFF_ROW);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(sm + Lay::OFF_ABORT);

  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xFFFFFFFFu, tid >> 5, 0);  // (the same in every lane, and known to be)
  const int slice = warp / RG, rg = warp % RG;
  const int fg = lane >> 2, ft = lane & 3;  // fragment row and column pair
  uint64_t *full = reinterpret_cast<uint64_t *>(sm + Lay::OFF_FULL) + slice * ST;
  uint64_t *empty = reinterpret_cast<uint64_t *>(sm + Lay::OFF_EMPTY) + slice * ST;
  // the group copied into each stage, twice, and 1 if its page is bad
  volatile int *s_copied = reinterpret_cast<volatile int *>(sm + Lay::OFF_COPIED) + slice * ST;
  uint8_t *ring = sm + slice * ST * Lay::G_BYTES;

  const unsigned C = p.cluster, rank = C > 1 ? cluster_rank() : 0;
  const int unit = blockIdx.x / C;
  const int mt = unit % p.m_tiles, kvh = (unit / p.m_tiles) % p.Hkv, b = unit / p.m_tiles / p.Hkv;
  const bool reports = kvh == 0 && mt == 0 && rank == 0;

  const bool layout_ok = (smem_u32(sm) & 1023u) == 0;  // 128-byte-swizzled boxes
  if (lane == 0 && rg == 0) {
    for (int i = 0; i < ST; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], RG);
      s_copied[i] = -2;
    }
    fence_barrier_init();
  }
  // the place of each of the CTA's rows in q and out, in heads (-1: past the unit's rows)
  if (tid < RB) {
    const int R = mt * RB + tid, node = R / p.G;
    s_row[tid] = R < p.M ? (b * p.N + node) * p.Hq + kvh * p.G + R - node * p.G : -1;
  }
  if (tid == 0) *abort_flag = 0;
  wait_previous();
  int L = p.prefix_len[b];
  if (tid < kMaxNodes) s_par[tid] = tid < p.N ? tree_parent(p.tree, b, tid) : -1;
  __syncthreads();
  // query rows as B operands, on their way before the first keys
  uint8_t *s_q = sm + Lay::OFF_Q;
#pragma unroll
  for (int u = tid; u < RB * (D / 8); u += kWinThreads) {
    const int r = u / (D / 8), c = u % (D / 8), row = s_row[r];
    cp_async_16(s_q + (c >> 3) * (RB * 128) + sw128_offset(r, c & 7),
                static_cast<const bf16 *>(p.q) + (size_t)max(row, 0) * D + 8 * c, row >= 0);
  }
  cp_async_commit();
  if (L < 0 || L > p.cap) {
    if (reports && tid == 0) set_status(p.status, SV_DEV_BAD_PREFIX);
    L = L < 0 ? 0 : p.cap;
  }
  const int lo_root = window_first(L, p.window);
  const int first = p.block_table ? lo_root & ~(kWinGroup - 1) : lo_root;
  const int n_sinks = min(p.sinks, first);
  // groups: tree nodes, sinks before the window, window
  const int gt = (p.N + kWinGroup - 1) / kWinGroup, gs = gt + (n_sinks + kWinGroup - 1) / kWinGroup;
  const int groups = gs + (L - first + kWinGroup - 1) / kWinGroup;
  const int per = (groups + (int)C - 1) / (int)C;
  const int g0 = min((int)rank * per, groups), g1 = min(g0 + per, groups);
  const int n = g1 - g0 > slice ? (g1 - g0 - slice + KS - 1) / KS : 0;  // this slice's groups

  // ---- copies: a slice's warp issues its groups' K and V; of two warps each does so for every other
  // group
  const uint64_t stream_policy = l2_policy_evict_first(), tree_policy = l2_policy_evict_normal();
  int desc = -1;  // lane i: row of group (32 k + i) of this slice, k the batch being issued
  auto locate = [&](int i) -> int {
    const int gi = g0 + slice + KS * i;
    if (i >= n) return -1;
    if (gi < gt) return b * p.N + kWinGroup * gi;
    const int pos = gi < gs ? kWinGroup * (gi - gt) : first + kWinGroup * (gi - gs);
    if (!p.block_table) return b * p.Lmax + pos;
    const int blk = p.block_table[(size_t)b * p.max_blocks + pos / p.block_size];
    if (blk < 0 || blk >= p.num_blocks) {
      set_status(p.status, SV_DEV_BAD_BLOCK);
      return -1;
    }
    return blk * p.block_size + pos % p.block_size;
  };
  // (one lane) group i, whose rows start at `row`, into stage st; none if the page is bad
  auto copy = [&](int i, int row, bool tree, int st) {
    s_copied[st] = 2 * i + (row < 0);
    if (row < 0) {
      mbar_arrive(&full[st]);
      return;
    }
    uint8_t *dst = ring + st * Lay::G_BYTES;
    const uint64_t policy = tree ? tree_policy : stream_policy;
    mbar_expect_tx(&full[st], Lay::G_BYTES);
    tma_load_4d_hint(dst, tree ? &p.tm_kt : &p.tm_kc, 0, row, 0, kvh, &full[st], policy);
    tma_load_4d_hint(dst + Lay::K_BYTES, tree ? &p.tm_vt : &p.tm_vc, 0, row, 0, kvh, &full[st], policy);
  };
  auto mine = [&](int i) { return RG == 1 || (i & 1) == rg; };
  // group i of the slice into stage st, which is free once its last group's barrier `empty` has
  // passed the parity
  auto issue = [&](int i, int st, int parity) {
    if ((i & 31) == 0) desc = locate(i + lane);
    if (!mine(i)) return;
    const int row = __shfl_sync(0xFFFFFFFFu, desc, i & 31);
    const bool tree = g0 + slice + KS * i < gt;
    if (elect_one() && (RG == 1 || parity < 0 || limited_wait(&empty[st], parity, abort_flag, p))) copy(i, row, tree, st);
    __syncwarp();
  };
  // The first groups, one after another so that the first one is whole soon (2048 units of 32 rows,
  // window 1025, 169 us against 176 with a lane each); with a lane each only for 33 to 48 rows (512
  // units, window 4097, 179 us against 185; 256 units of 64 rows, window 513, 23.8 against 24.9).
  static_assert(ST <= 32, "the first groups are one batch");
  if (layout_ok) {
    if (RG == 2 && NT < 4) {
      desc = locate(lane);
      if (lane < min(ST, n) && mine(lane)) copy(lane, desc, g0 + slice + KS * lane < gt, lane);
      __syncwarp();
    } else {
      for (int i = 0; i < min(ST, n); ++i) issue(i, i, -1);
    }
  }

  // ---- what each row sees
  if (tid < RB) {
    const int R = mt * RB + tid;
    uint64_t anc = 0;
    int lo = 0;
    if (R < p.M) {
      int depth;
      if (!tree_walk(s_par, R / p.G, &anc, &depth) && kvh == 0 && rank == 0) set_status(p.status, SV_DEV_BAD_TREE);
      lo = window_first(L + depth, p.window);
      anc = window_ancestors(anc, L, p.window, p.sinks);
    }
    s_anc[tid] = anc;
    s_lo[tid] = lo;
  }
  cp_async_wait<0>();
  __syncthreads();
  // Every row sees every key of the groups [plain0, plain1) of this slice: inside the window of all
  // rows (none starts later than the deepest possible node's), before the prefix's end.
  const int lo_last = window_first(L + p.N - 1, p.window);
  const int plain0 = max(0, gs + (lo_last - first + kWinGroup - 1) / kWinGroup - g0 - slice + KS - 1) / KS;
  const int plain1 = max(0, gs + (L - first) / kWinGroup - g0 - slice + KS - 1) / KS;

  float o[DT][NT][4];
#pragma unroll
  for (int d = 0; d < DT; ++d)
#pragma unroll
    for (int j = 0; j < NT; ++j) o[d][j][0] = o[d][j][1] = o[d][j][2] = o[d][j][3] = 0.f;
  float m[NT][2], l[NT][2];
#pragma unroll
  for (int j = 0; j < NT; ++j) m[j][0] = m[j][1] = kWinNone, l[j][0] = l[j][1] = 0.f;

  const float sc = p.scale_log2;
  // this lane's row of a group for the two kinds of fragment loads, and its 16-byte chunks
  const int k_row = lane & 15, k_chunk = lane >> 4;
  const int v_row = (lane & 7) + ((lane >> 4) << 3), v_chunk = (lane >> 3) & 1;
  // 16-byte chunk 2q + chunk of a 64-column block, q = 0..3: the swizzle is an exclusive or, so
  // the four offsets differ by constants in bits 5 and 6
  const uint32_t k_off = sw128_offset(k_row, k_chunk), v_off = sw128_offset(v_row, v_chunk);
  const uint32_t ring_addr = smem_u32(ring);
  // query rows as B operands: 8 rows of 8-column step j, 16-byte chunks 2k + 0..3 (two 16-column
  // steps in one load), the same exclusive-or swizzle
  const uint32_t q_row = (uint32_t)(rg * 8 * NT + (lane & 7));
  const uint32_t q_addr = smem_u32(s_q) + q_row * 128u + ((((uint32_t)lane >> 3) ^ (q_row & 7)) << 4);
  auto load_q = [&](int k, uint32_t (&q)[NT][4]) {
#pragma unroll
    for (int j = 0; j < NT; ++j) ldsm_x4(q[j], (q_addr ^ ((k & 2) << 5)) + (k >> 2) * (RB * 128) + j * 1024);
  };
  // held in registers where there is room for them, else loaded for each group
  constexpr bool kHold = RG == 1 || NT < 4;
  uint32_t held[kHold ? DT / 2 : 1][NT][4];
  if constexpr (kHold) {
#pragma unroll
    for (int k = 0; k < DT; k += 2) load_q(k, held[k / 2]);
  }
  int done = 0;
  int st = 0, phase = 0;  // the stage of group i and the parity of its use

  float s[NT][4];      // the scores of the group whose weights come next, then their exponents
  uint32_t pb[NT][2];  // its weights
  // half h of the weights of 8-column step j
  auto weigh = [&](int j, int h) {
    const float x0 = ex2_approx(s[j][2 * h]), x1 = ex2_approx(s[j][2 * h + 1]);
    l[j][0] += x0;
    l[j][1] += x1;
    pb[j][h] = transpose_8x8(pack_bf16x2(x0, x1));
  };
  // Products of a group's keys with the query rows, each step's operands loaded a step ahead; with
  // WEIGH the weights of the group before, between the products.  (512 units of 104 rows, window 4097:
  // 566 us with one group after another, 525 with two groups side by side, 481 this way.)
  auto scores = [&](auto weigh_too, uint32_t stage, float (&t)[NT][4]) {
    constexpr bool WEIGH = decltype(weigh_too)::value;
    auto load_k = [&](int k, uint32_t (&a)[4]) {
      ldsm_x4(a, stage + (k_off ^ ((k & 3) << 5)) + (k >> 2) * (kWinGroup * 128));
    };
    uint32_t a[2][4], q[2][NT][4];
    if constexpr (!kHold) load_q(0, q[0]);
    load_k(0, a[0]);
#pragma unroll
    for (int k = 0; k < DT; ++k) {
      if (k + 1 < DT) load_k(k + 1, a[(k + 1) & 1]);
      if (!kHold && k % 2 == 0 && k + 2 < DT) load_q(k + 2, q[(k / 2 + 1) & 1]);
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        const uint32_t *b = kHold ? held[kHold ? k / 2 : 0][j] : q[(k / 2) & 1][j];
        if (k == 0) mma_first(t[j], a[0], b[0], b[1]);
        else mma_bf16_16816(t[j], a[k & 1], b[2 * (k & 1)], b[2 * (k & 1) + 1]);
      }
      if constexpr (WEIGH) {
#pragma unroll
        for (int u = k * 2 * NT / DT; u < (k + 1) * 2 * NT / DT; ++u) weigh(u >> 1, u & 1);
      }
    }
  };
  // Products of the weights with the group's V.
  auto outputs = [&](uint32_t stage) {
    auto load_v = [&](int d, uint32_t (&a)[4]) {
      ldsm_x4_trans(a, stage + Lay::K_BYTES + (v_off ^ ((d & 3) << 5)) + (d >> 2) * (kWinGroup * 128));
    };
    uint32_t a[2][4];
    load_v(0, a[0]);
#pragma unroll
    for (int d = 0; d < DT; ++d) {
      if (d + 1 < DT) load_v(d + 1, a[(d + 1) & 1]);
#pragma unroll
      for (int j = 0; j < NT; ++j) mma_bf16_16816(o[d][j], a[d & 1], pb[j][0], pb[j][1]);
    }
  };
  // What the rows do not see of group i goes from its scores (all of it if its page is bad).
  auto mask = [&](int i, uint32_t stage, bool bad) {
    if (!bad && i >= plain0 && i < plain1) return;
    const int gi = g0 + slice + KS * i;
    const int base = gi < gs ? kWinGroup * (gi < gt ? gi : gi - gt) : first + kWinGroup * (gi - gs);
    const bool tree = gi < gt;
    const int end = bad ? 0 : (tree ? p.N : (gi < gs ? n_sinks : L));
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int r = rg * 8 * NT + 8 * j + 2 * ft + e, key = base + fg;
        bool see0, see1;
        if (tree) {
          const uint32_t seen = (uint32_t)(s_anc[r] >> base) >> fg;
          see0 = seen & 1u;
          see1 = seen & 256u;
        } else {
          const int lo = s_lo[r];
          see0 = key < end && (key >= lo || key < p.sinks);
          see1 = key + 8 < end && (key + 8 >= lo || key + 8 < p.sinks);
        }
        if (!see0) s[j][e] = -INFINITY;
        if (!see1) s[j][e + 2] = -INFINITY;
      }
    // V rows that no row sees may hold anything: zero them, so that 0 * V stays 0
    const int key = base + k_row;
    const bool live = key < end && (tree || key >= lo_root || key < p.sinks);
    if (__all_sync(0xFFFFFFFFu, live)) return;
    if (!live) {
      uint8_t *sv = ring + (stage - ring_addr) + Lay::K_BYTES;
#pragma unroll
      for (int c = 0; c < D / 16; ++c) {
        const int ch = k_chunk * (D / 16) + c;
        *reinterpret_cast<uint4 *>(sv + (ch >> 3) * (kWinGroup * 128) + sw128_offset(k_row, ch & 7)) =
            make_uint4(0, 0, 0, 0);
      }
    }
    fence_proxy_async_smem();  // before the next copy into this stage
    __syncwarp();
  };
  // The weights are taken against a maximum of each row that need not be the latest: only
  // when a score passes it by more than 2^8 (or there is none yet) is it brought up to date
  // over the warp's keys, and the sums and outputs with it.  Then no exchange between
  // lanes is needed but one vote.
  auto limits = [&]() {
    float x[NT][4], top = -INFINITY;
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        x[j][e] = fmaf(s[j][e], sc, -m[j][e & 1]);
        top = fmaxf(top, x[j][e]);
      }
    if (!__any_sync(0xFFFFFFFFu, top > kWinRescale)) {
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[j][e] = x[j][e];
      return;
    }
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      float w[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float y = fmaxf(s[j][e], s[j][e + 2]);
        y = fmaxf(y, __shfl_xor_sync(0xFFFFFFFFu, y, 4));
        y = fmaxf(y, __shfl_xor_sync(0xFFFFFFFFu, y, 8));
        y = fmaxf(y, __shfl_xor_sync(0xFFFFFFFFu, y, 16));
        y = fmaxf(y * sc, m[j][e]);
        w[e] = ex2_approx(m[j][e] - y);
        m[j][e] = y;
        l[j][e] *= w[e];
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) s[j][e] = fmaf(s[j][e], sc, -m[j][e & 1]);
#pragma unroll
      for (int d = 0; d < DT; ++d) {
        o[d][j][0] *= w[0];
        o[d][j][1] *= w[1];
        o[d][j][2] *= w[0];
        o[d][j][3] *= w[1];
      }
    }
  };
  auto arrived = [&](int at, int par) -> bool {
    return __all_sync(0xFFFFFFFFu, limited_wait(&full[at], par, abort_flag, p));
  };
  // the stage of group i - back is filled again with group i - back + ST
  auto refill = [&](int i, int back) {
    if (i < back || i - back + ST >= n) return;
    issue(i - back + ST, st >= back ? st - back : st - back + ST, st >= back ? phase : phase ^ 1);
  };
  auto next_stage = [&]() {  // done with the stage
    __syncwarp();            // every lane is
    if (RG > 1 && lane == 0) mbar_arrive(&empty[st]);
    if (++st == ST) st = 0, phase ^= 1;
  };
  if constexpr (kHold) {
    for (int i = 0; layout_ok && i < n; ++i) {
      // (two warps that share a slice need not be done with the previous group at the same time)
      refill(i, RG);
      if (!arrived(st, phase)) break;
      done = i + 1;
      if ((s_copied[st] & 1) == 0) {
        const uint32_t stage = ring_addr + st * Lay::G_BYTES;
        scores(std::false_type{}, stage, s);
        mask(i, stage, false);
        limits();
#pragma unroll
        for (int u = 0; u < 2 * NT; ++u) weigh(u >> 1, u & 1);
        outputs(stage);
      }
      next_stage();
    }
  } else if (layout_ok && n > 0 && arrived(0, 0)) {
    // the scores of a group are computed between the weights of the one before
    done = 1;
    scores(std::false_type{}, ring_addr, s);
    mask(0, ring_addr, (s_copied[0] & 1) != 0);
    limits();
    for (int i = 0; i < n; ++i) {
      const uint32_t stage = ring_addr + st * Lay::G_BYTES;
      const int st1 = st + 1 == ST ? 0 : st + 1;
      const uint32_t stage1 = ring_addr + st1 * Lay::G_BYTES;
      if (i + 1 == n) {
#pragma unroll
        for (int u = 0; u < 2 * NT; ++u) weigh(u >> 1, u & 1);
        outputs(stage);
        break;
      }
      if (!arrived(st1, st1 == 0 ? phase ^ 1 : phase)) break;
      done = i + 2;
      const bool bad = (s_copied[st1] & 1) != 0;
      float t[NT][4];
      scores(std::true_type{}, stage1, t);
      outputs(stage);
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[j][e] = t[j][e];
      refill(i, 1);  // (by now the other warp of the slice is done with that stage too)
      next_stage();
      mask(i + 1, stage1, bad);
      limits();
    }
  }
  if (done < n && layout_ok) {
    // a wait gave up: let this warp's copies in flight (those that were made) land before the shared
    // memory is used again
    *abort_flag = 1;
    const unsigned long long t0 = global_ns();
    for (int k = 0; k < ST; ++k) {
      const int i = s_copied[k] >> 1;
      while (i >= done && mine(i) && !mbar_try_wait(&full[k], (i / ST) & 1) && global_ns() - t0 < kWaitLimitNs) {
      }
    }
  }

  // ---- merge, in units of 16 dimensions of 8 rows as they stand in a warp's registers (one float4
  // per lane).  A slice takes DT / KS of the 16-dimension tiles and gets them from the others.
  constexpr int DO = Lay::DO, U = Lay::UNITS;
  float4 *part = reinterpret_cast<float4 *>(sm);      // [KS taker][KS - 1][RG][DO][NT][32]
  float4 *joined = reinterpret_cast<float4 *>(sm + Lay::OFF_JOIN);  // [C][units of this CTA][32]
  float *c_m = reinterpret_cast<float *>(joined + (U + 8) * 32), *c_l = c_m + 8 * RB;  // [C][RB]
  // Done with the ring.  (Room of its own for what the others write and an arrival at the start gain
  // nothing.)
  if (C > 1) cluster_arrive();
#pragma unroll
  for (int j = 0; j < NT; ++j)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      l[j][e] += __shfl_xor_sync(0xFFFFFFFFu, l[j][e], 4);
      l[j][e] += __shfl_xor_sync(0xFFFFFFFFu, l[j][e], 8);
      l[j][e] += __shfl_xor_sync(0xFFFFFFFFu, l[j][e], 16);
      if (fg == 0) {
        const int r = rg * 8 * NT + 8 * j + 2 * ft + e;
        s_m[slice * RB + r] = m[j][e];
        s_l[slice * RB + r] = l[j][e];
      }
    }
  __syncthreads();  // (and every slice is done with its ring)
  float w[NT][2];   // this slice's weights against the CTA's maximum
#pragma unroll
  for (int j = 0; j < NT; ++j)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int r = rg * 8 * NT + 8 * j + 2 * ft + e;
      float top = kWinNone;
#pragma unroll
      for (int k = 0; k < KS; ++k) top = fmaxf(top, s_m[k * RB + r]);
      w[j][e] = ex2_approx(m[j][e] - top);
    }
  auto scaled = [&](int d, int j) {
    return make_float4(o[d][j][0] * w[j][0], o[d][j][1] * w[j][1], o[d][j][2] * w[j][0], o[d][j][3] * w[j][1]);
  };
  auto place = [&](int taker, int k, int d, int j) {
    return part + ((((taker * (KS - 1) + k) * RG + rg) * DO + d % DO) * NT + j) * 32 + lane;
  };
#pragma unroll
  for (int d = 0; d < DT; ++d) {
    const int taker = d / DO;
    if (taker != slice) {
#pragma unroll
      for (int j = 0; j < NT; ++j) *place(taker, slice < taker ? slice : slice - 1, d, j) = scaled(d, j);
    }
  }
  float top = kWinNone, sum = 0.f;
  if (tid < RB) {
#pragma unroll
    for (int k = 0; k < KS; ++k) top = fmaxf(top, s_m[k * RB + tid]);
#pragma unroll
    for (int k = 0; k < KS; ++k) sum += ex2_approx(s_m[k * RB + tid] - top) * s_l[k * RB + tid];
    if (C == 1) s_inv[tid] = sum > 0.f ? 1.f / sum : 0.f;
  }
  __syncthreads();
  // a unit's final values to memory: rows 2 ft and 2 ft + 1 of dimensions fg and fg + 8 become, by
  // a transpose and an exchange of neighbours, four dimensions of row fg
  auto emit = [&](int d, int row, float4 v) {
    const uint32_t a = transpose_8x8(pack_bf16x2(v.x, v.y)), c = transpose_8x8(pack_bf16x2(v.z, v.w));
    const bool odd = lane & 1;
    const uint32_t other = __shfl_xor_sync(0xFFFFFFFFu, odd ? a : c, 1);
    if (row >= 0)
      *reinterpret_cast<uint2 *>(static_cast<bf16 *>(p.out) + (size_t)row * D + 16 * d + (odd ? 6 + 2 * ft : 2 * ft)) =
          odd ? make_uint2(other, c) : make_uint2(a, other);
  };
  const int shift = 31 - __clz((int)C), local = (U + (int)C - 1) >> shift;  // units of a CTA
  if (C > 1) {
    cluster_wait();  // every CTA of the cluster is done with its ring
    if (tid < RB)
      for (unsigned c = 0; c < C; ++c) {
        remote_store(remote_address(c_m + rank * RB + tid, c), top);
        remote_store(remote_address(c_l + rank * RB + tid, c), sum);
      }
  }
  float inv[NT][2];
  int rows[NT];
  if (C == 1) {
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      const int r0 = rg * 8 * NT + 8 * j;
      rows[j] = s_row[r0 + fg];
      inv[j][0] = s_inv[r0 + 2 * ft];
      inv[j][1] = s_inv[r0 + 2 * ft + 1];
    }
  }
#pragma unroll
  for (int d = 0; d < DT; ++d) {
    if (d / DO != slice) continue;
    float4 x[NT][KS - 1];
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int k = 0; k < KS - 1; ++k) x[j][k] = *place(d / DO, k, d, j);
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      float4 v = scaled(d, j);
#pragma unroll
      for (int k = 0; k < KS - 1; ++k) {
        v.x += x[j][k].x;
        v.y += x[j][k].y;
        v.z += x[j][k].z;
        v.w += x[j][k].w;
      }
      if (C == 1) {
        emit(d, rows[j], make_float4(v.x * inv[j][0], v.y * inv[j][1], v.z * inv[j][0], v.w * inv[j][1]));
      } else {
        const int u = (rg * DT + d) * NT + j;
        remote_store(remote_address(joined + ((int)rank * local + (u >> shift)) * 32 + lane, u & (C - 1)), v);
      }
    }
  }
  if (C > 1) {
    // each CTA joins its units of the whole cluster; nobody looks into another CTA any more
    cluster_sync();
    // the CTAs' weights of a row, for all rows first where a warp joins more than one unit
    constexpr bool kTable = U > 16;
    auto weights_of = [&](int r, float2 (&wc)[8]) {  // of rows r and r + 1
      float2 sums[8], top = make_float2(kWinNone, kWinNone), total = make_float2(0.f, 0.f);
#pragma unroll
      for (int c = 0; c < 8; ++c) {
        wc[c] = top;
        sums[c] = total;
        if (c < (int)C) {
          wc[c] = *reinterpret_cast<const float2 *>(c_m + c * RB + r);
          sums[c] = *reinterpret_cast<const float2 *>(c_l + c * RB + r);
        }
      }
#pragma unroll
      for (int c = 0; c < 8; ++c) top = make_float2(fmaxf(top.x, wc[c].x), fmaxf(top.y, wc[c].y));
#pragma unroll
      for (int c = 0; c < 8; ++c) {
        wc[c] = make_float2(ex2_approx(wc[c].x - top.x), ex2_approx(wc[c].y - top.y));
        total = make_float2(fmaf(wc[c].x, sums[c].x, total.x), fmaf(wc[c].y, sums[c].y, total.y));
      }
      const float i0 = total.x > 0.f ? 1.f / total.x : 0.f, i1 = total.y > 0.f ? 1.f / total.y : 0.f;
#pragma unroll
      for (int c = 0; c < 8; ++c) wc[c] = make_float2(wc[c].x * i0, wc[c].y * i1);
    };
    float2 wc[8];
    if (kTable) {
      if (tid < RB / 2) {
        weights_of(2 * tid, wc);
#pragma unroll
        for (int c = 0; c < 8; ++c)
          if (c < (int)C) *reinterpret_cast<float2 *>(c_m + c * RB + 2 * tid) = wc[c];
      }
      __syncthreads();
    }
    for (int i = warp; i < local; i += kWinThreads / 32) {
      const int u = (i << shift) + (int)rank;
      if (u >= U) break;
      const int j = u % NT, d = u / NT % DT, r0 = u / NT / DT * 8 * NT + 8 * j;
      float4 y[8];
#pragma unroll
      for (int c = 0; c < 8; ++c)
        if (c < (int)C) y[c] = joined[(c * local + i) * 32 + lane];
      if (!kTable) weights_of(r0 + 2 * ft, wc);
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int c = 0; c < 8; ++c) {
        if (c >= (int)C) break;
        if (kTable) wc[c] = *reinterpret_cast<const float2 *>(c_m + c * RB + r0 + 2 * ft);
        v.x = fmaf(wc[c].x, y[c].x, v.x);
        v.y = fmaf(wc[c].y, y[c].y, v.y);
        v.z = fmaf(wc[c].x, y[c].z, v.z);
        v.w = fmaf(wc[c].y, y[c].w, v.w);
      }
      emit(d, s_row[r0 + fg], v);
    }
  }
  if (tid == 0) {
    if (!layout_ok) set_status(p.status, SV_DEV_LAYOUT);
    else if (*abort_flag) set_status(p.status, SV_DEV_TIMEOUT);
  }
}

template <int D, int NT, int RG>
cudaError_t launch_window_typed(const WinParams &p, long long ctas, cudaStream_t s) {
  using Lay = WinLayout<D, NT, RG>;
  static std::atomic<bool> attr[64];
  int dev = 0;
  cudaGetDevice(&dev);
  auto kern = window_attn_kernel<D, NT, RG>;
  if (dev < 0 || dev >= 64 || !attr[dev].load()) {
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Lay::SMEM);
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < 64) attr[dev].store(true);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)ctas);
  cfg.blockDim = dim3(kWinThreads);
  cfg.dynamicSmemBytes = Lay::SMEM;
  cfg.stream = s;
  cudaLaunchAttribute at[2];
  at[0] = close_launch();
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = (unsigned)p.cluster;
  at[1].val.clusterDim.y = 1;
  at[1].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = p.cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kern, p);
}

template <int D>
cudaError_t launch_window_d(const WinParams &p, int nt, int rg, long long ctas, cudaStream_t s) {
  if (rg == 2) return nt == 3 ? launch_window_typed<D, 3, 2>(p, ctas, s) : launch_window_typed<D, 4, 2>(p, ctas, s);
  if (nt == 1) return launch_window_typed<D, 1, 1>(p, ctas, s);
  if (nt == 2) return launch_window_typed<D, 2, 1>(p, ctas, s);
  return nt == 3 ? launch_window_typed<D, 3, 1>(p, ctas, s) : launch_window_typed<D, 4, 1>(p, ctas, s);
}

// Rows of a CTA: up to four 8-column steps per warp, or up to four per each of a slice's two warps.
// Few rows per CTA make short chains and many CTAs, which read the same K and V from L2; many rows
// read them once.  Fitted to measurements (D = 128, contiguous caches, 8 to 128 units of 32 to 512 rows,
// windows 17 to 4097, root mean square error 5 %; D = 64 goes by the same figures, its bytes counted
// twice over): a CTA takes `start` us and `group` us for each of its groups, 1.16 times
// that with two CTAs per SM.  8 units of 64 rows, window 4097, in tiles of 16 rows 12.1 us against
// 18.3 in one; 128 units of 208 rows, window 4097, in tiles of 32 rows 177 against 223 in tiles of
// 64; 512 rows, window 513, 114 against 90.
struct WinForm {
  int nt, rg;
  double start, group;
};
constexpr WinForm kWinForms[] = {{4, 2, 5.9, 0.363}, {3, 2, 4.8, 0.281}, {4, 1, 5.5, 0.179},
                                 {3, 1, 4.6, 0.145}, {2, 1, 3.7, 0.126}, {1, 1, 2.7, 0.112}};
struct WinPlan {
  int nt, rg, m_tiles, cluster;
  double us;
};

// M rows against `groups` groups of keys for each of `kv_units` sequences and KV heads.
WinPlan window_plan(long long kv_units, int M, int groups, int num_sms) {
  WinPlan plan{};
  const double sms = num_sms, moved = (double)kv_units * groups * kWinGroup * 512 * 1e-6;  // K and V, MB
  for (const WinForm &f : kWinForms) {
    const int rows = 8 * f.nt * f.rg;
    // no more rows than the unit's, in whole steps (three or four for two warps)
    if (f.rg == 2 ? M <= (f.nt == 4 ? 48 : 32) : rows >= M + 8) continue;
    const int tiles = (M + rows - 1) / rows;
    const long long units = kv_units * tiles, slots = 2ll * num_sms;
    // CTAs per unit: waves of resident CTAs times the length of one, which costs about 16 groups
    // (its start and merge) beside its share of the window's groups: 512 units of 32 rows, window
    // 4097, go without clusters, 156 us against 181 with clusters of four.  (Clusters of 16 gain
    // little on the longest windows and start later: 8 units of 4 rows, window 1024, 0.6 us more; 16
    // such clusters find no room together, 25 us against 13.)
    long long best = 0;
    int cluster = 1;
    for (int c = 1; c <= 8; c *= 2) {
      const long long cost = (units * c + slots - 1) / slots * ((groups + c - 1) / c + 16);
      if (c == 1 || cost < best) {
        best = cost;
        cluster = c;
      }
    }
    const double load = (double)units * cluster / (2 * sms);
    const double waves = load <= 0.5 ? 1 : 1.16 * (load <= 3 ? std::ceil(load) : load + 0.5);
    const double chains = waves * (f.start + f.group * ((groups + cluster - 1) / cluster));
    const double us = 1.6 + (cluster > 1 ? 1.3 : 0) + std::max(chains, std::max(moved / 5.8, moved * tiles / 18.2));
    // (more tiles have to be worth it)
    if (plan.us == 0 || us < 0.97 * plan.us) plan = {f.nt, f.rg, tiles, cluster, us};
  }
  return plan;
}

}  // namespace

// The tensor-core kernel pads a unit's rows to 128 or 256 and pays more for a unit's start and
// for the launch, but takes long windows of many rows at twice the rate.  As fitted to measurements
// (us; D = 128, contiguous caches, 128 to 2048 units, 40 to 512 rows, windows 17 to 4097):
//   13 + units tiles / SMs (6 + 1.45 key tiles) + 2 SMs / units      (2.55 for 256 rows)
// e.g. 128 units of 104 rows: window 129 13 us here against 21, window 1025 36 against 33; 512 units
// of 64 rows: 24 against 39, 69 against 87; 8 units of 208 rows, window 4097: 20 against 85.
// Up to 32 rows this kernel runs at the memory's rate: 2048 units, window 1025: 172 against 270.
bool window_prefers_tc(int B, int N, int Hq, int Hkv, int span, int num_sms) {
  const int M = N * (Hq / Hkv);
  if (M <= 32) return false;
  const double units = (double)B * Hkv, sms = num_sms;
  const double here = window_plan((long long)B * Hkv, M, span / kWinGroup + N / kWinGroup + 2, num_sms).us;
  const double tiles = span / 128 + 2;
  const double there = 13 + units * ((M + 255) / 256) / sms * (6 + (M > 128 ? 2.55 : 1.45) * tiles) + 2 * sms / units;
  return there < here;
}

cudaError_t launch_window_attention(const AttnParams &a, int num_sms, cudaStream_t s) {
  WinParams p{};
  const long long rows = a.block_table ? (long long)a.num_blocks * a.block_size
                                       : (long long)a.B * (a.Lmax > 0 ? a.Lmax : 1);
  if (!tma_rows_map(&p.tm_kt, a.k_tree, a.D, a.Hkv, (long long)a.B * a.N, kWinGroup) ||
      !tma_rows_map(&p.tm_vt, a.v_tree, a.D, a.Hkv, (long long)a.B * a.N, kWinGroup) ||
      !tma_rows_map(&p.tm_kc, a.cache_k, a.D, a.Hkv, rows, kWinGroup) ||
      !tma_rows_map(&p.tm_vc, a.cache_v, a.D, a.Hkv, rows, kWinGroup))
    return cudaErrorInvalidValue;
  p.q = a.q;
  p.out = a.out;
  p.prefix_len = a.prefix_len;
  p.block_table = a.block_table;
  p.status = a.status;
  p.B = a.B;
  p.N = a.N;
  p.Hq = a.Hq;
  p.Hkv = a.Hkv;
  p.G = a.G;
  p.M = a.M;
  p.Lmax = a.Lmax;
  p.block_size = a.block_size;
  p.max_blocks = a.max_blocks;
  p.num_blocks = a.num_blocks;
  p.cap = a.cap;
  p.window = a.window;
  p.sinks = a.sinks;
  p.scale_log2 = a.scale_log2;
  p.tree = a.tree;
  p.wait_ns = a.wait_ns;
  p.try_ns = (unsigned)std::min<unsigned long long>(a.wait_ns, kWinTryNs);
  const int span = a.window - 1 < a.cap ? a.window - 1 : a.cap;
  const WinPlan plan = window_plan((long long)a.B * a.Hkv, a.M, span / kWinGroup + (a.N + a.sinks) / kWinGroup + 2, num_sms);
  p.m_tiles = plan.m_tiles;
  p.cluster = plan.cluster;
  const long long units = (long long)a.B * a.Hkv * p.m_tiles;
  const long long ctas = units * p.cluster;
  if (ctas > INT32_MAX) return cudaErrorInvalidValue;
  return a.D == 128 ? launch_window_d<128>(p, plan.nt, plan.rg, ctas, s) : launch_window_d<64>(p, plan.nt, plan.rg, ctas, s);
}

}  // namespace sv
