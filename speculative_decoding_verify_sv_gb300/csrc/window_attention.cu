// Tree attention over a sliding window with sinks for units of few query rows (sm_103a, bf16).
//
// Node n of sequence b stands at P = L_b + depth(n); its keys are the prefix positions p with
// P - p < window or p < sinks, and the nodes of its root path by the same rule.  A unit is a
// sequence and KV head: its M = N * G query rows (tree nodes x group heads) against
//   the tree's N nodes, the sinks before the window, and [first, L_b),
// first = L_b - window + 1 being the earliest position that a row's window reaches (rounded
// down to 16 in a paged cache).  These keys are cut into groups of 16, none of which crosses a
// page.
//
// With few rows the work is a stream of K and V: what counts is that loads are always in
// flight and that units, which a window keeps short, begin and end without gaps.  So nothing
// in the main loop waits for another warp: each slice of a CTA (one warp; two with more than
// 32 rows, which then share a slice's rows) takes every KS-th group, has a ring of its own
// in shared memory, issues its own TMA copies (16 rows per box, several groups ahead) and
// keeps its own running maximum, sum and output in registers.  Two CTAs share an SM, so one
// streams while the other starts or ends.
//
// The products are taken transposed, S^T = K Q^T and O^T = V^T P^T: keys and head
// dimensions fill the 16-row side of the matrix instruction and the query rows its 8-column
// side, so that 4 rows (one token, 4 group heads) cost one 8-column step and 20 rows cost
// three, where a 128-row tcgen05 tile would be padded to 128.  P^T goes from accumulator to
// operand layout by an 8x8 transpose in registers, rounded to bf16 (off by at most 2^-8 of each
// weight; the sum is of the unrounded ones); scores, weights, sums and outputs are fp32.
//
// Bound by HBM for many units: 256 ragged requests of 5 nodes, 32:8 heads of 128, window 1024 in pages
// of 16, 177 us, 6.1 TB/s, 90 % of the measured copy rate (the 128-row kernel 268 us); by latency
// for few: one token of one request, window 1024, 6.6 us (49).
//
// The slices merge in shared memory by weights 2^(m_slice - m).  Few long units: a cluster of
// up to 8 CTAs shares a unit's groups and merges through distributed shared memory, without a
// workspace or a second launch.
#include <atomic>
#include <cfloat>
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
  static constexpr int OS = D + 4;              // row stride of the merged outputs (floats): no bank conflicts
  static constexpr int OFF_Q = RING;            // query rows [RB][D], 128-byte swizzle per 64 columns
  static constexpr int OFF_FULL = OFF_Q + RB * D * 2;
  static constexpr int OFF_EMPTY = OFF_FULL + KS * ST * 8;
  static constexpr int OFF_ANC = OFF_EMPTY + KS * ST * 8;
  static constexpr int OFF_M = OFF_ANC + RB * 8;        // [KS][RB]
  static constexpr int OFF_L = OFF_M + KS * RB * 4;     // [KS][RB]
  static constexpr int OFF_CM = OFF_L + KS * RB * 4;    // [RB] the CTA's maximum and sum
  static constexpr int OFF_CL = OFF_CM + RB * 4;
  static constexpr int OFF_LO = OFF_CL + RB * 4;        // [RB]
  static constexpr int OFF_ROW = OFF_LO + RB * 4;       // [RB]
  static constexpr int OFF_PAR = OFF_ROW + RB * 4;      // [64]
  static constexpr int OFF_BAD = OFF_PAR + kMaxNodes * 4;  // [KS][ST]
  static constexpr int OFF_ABORT = OFF_BAD + KS * ST * 4;
  static constexpr int SMEM = OFF_ABORT + 16;
  static_assert(KS * RB * OS * 4 <= RING, "the slices' outputs merge in the ring's room");
  static_assert(SMEM <= 113 * 1024, "two CTAs per SM");
};

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

template <int D, int NT, int RG>
__global__ void __launch_bounds__(kWinThreads, 2) window_attn_kernel(const __grid_constant__ WinParams p) {
  using Lay = WinLayout<D, NT, RG>;
  constexpr int KS = Lay::KS, KB = Lay::KB, ST = Lay::ST, RB = Lay::RB, OS = Lay::OS, DT = D / 16;
  extern __shared__ __align__(1024) uint8_t win_smem[];
  uint8_t *sm = win_smem;
  uint64_t *s_anc = reinterpret_cast<uint64_t *>(sm + Lay::OFF_ANC);
  float *s_m = reinterpret_cast<float *>(sm + Lay::OFF_M), *s_l = reinterpret_cast<float *>(sm + Lay::OFF_L);
  float *s_cm = reinterpret_cast<float *>(sm + Lay::OFF_CM), *s_cl = reinterpret_cast<float *>(sm + Lay::OFF_CL);
  int *s_lo = reinterpret_cast<int *>(sm + Lay::OFF_LO), *s_par = reinterpret_cast<int *>(sm + Lay::OFF_PAR);
  int *s_row = reinterpret_cast<int *>(sm + Lay::OFF_ROW);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(sm + Lay::OFF_ABORT);

  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xFFFFFFFFu, tid >> 5, 0);  // (the same in every lane, and known to be)
  const int slice = warp / RG, rg = warp % RG;
  const int fg = lane >> 2, ft = lane & 3;  // fragment row and column pair
  uint64_t *full = reinterpret_cast<uint64_t *>(sm + Lay::OFF_FULL) + slice * ST;
  uint64_t *empty = reinterpret_cast<uint64_t *>(sm + Lay::OFF_EMPTY) + slice * ST;
  volatile int *s_bad = reinterpret_cast<volatile int *>(sm + Lay::OFF_BAD) + slice * ST;
  uint8_t *ring = sm + slice * ST * Lay::G_BYTES;

  const unsigned C = p.cluster, rank = C > 1 ? cluster_rank() : 0;
  const int unit = blockIdx.x / C;
  const int mt = unit % p.m_tiles, kvh = (unit / p.m_tiles) % p.Hkv, b = unit / p.m_tiles / p.Hkv;
  const bool reports = kvh == 0 && mt == 0 && rank == 0;

  wait_previous();
  int L = p.prefix_len[b];
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

  // the place of each of the CTA's rows in q and out, in heads (-1: past the unit's rows)
  if (tid < RB) {
    const int R = mt * RB + tid, node = R / p.G;
    s_row[tid] = R < p.M ? (b * p.N + node) * p.Hq + kvh * p.G + R - node * p.G : -1;
  }
  if (tid < kMaxNodes) s_par[tid] = tid < p.N ? tree_parent(p.tree, b, tid) : -1;
  if (tid == 0) *abort_flag = 0;

  // ---- copies: a slice's warp issues its groups' K and V; two warps share that out
  constexpr bool kBoth = RG == 1;
  constexpr uint32_t kTx = kBoth ? Lay::G_BYTES : Lay::K_BYTES;
  const CUtensorMap *map_tree = rg == 0 ? &p.tm_kt : &p.tm_vt, *map_cache = rg == 0 ? &p.tm_kc : &p.tm_vc;
  const uint64_t stream_policy = l2_policy_evict_first();
  int desc = -1;  // lane i: row of group (32 k + i) of this slice, k the batch being issued
  auto locate = [&](int i) -> int {
    const int gi = g0 + slice + KS * i;
    if (i >= n) return -1;
    if (gi < gt) return b * p.N + kWinGroup * gi;
    const int pos = gi < gs ? kWinGroup * (gi - gt) : first + kWinGroup * (gi - gs);
    if (!p.block_table) return b * p.Lmax + pos;
    const int blk = __ldg(p.block_table + (size_t)b * p.max_blocks + pos / p.block_size);
    if (blk < 0 || blk >= p.num_blocks) {
      set_status(p.status, SV_DEV_BAD_BLOCK);
      return -1;
    }
    return blk * p.block_size + pos % p.block_size;
  };
  // group i of the slice into stage st, which is free once its last group's barrier `empty` has
  // passed the parity (-1: no group was there)
  auto issue = [&](int i, int st, int parity) {
    if ((i & 31) == 0) desc = locate(i + lane);
    const int row = __shfl_sync(0xFFFFFFFFu, desc, i & 31);
    const bool tree = g0 + slice + KS * i < gt;
    if (elect_one() && (kBoth || parity < 0 || mbar_wait(&empty[st], parity, abort_flag, p.wait_ns))) {
      s_bad[st] = row < 0;
      if (row < 0) {
        mbar_arrive(&full[st]);
      } else {
        uint8_t *dst = ring + st * Lay::G_BYTES + (kBoth ? 0 : rg * Lay::K_BYTES);
        mbar_expect_tx(&full[st], kTx);
#pragma unroll
        for (int kb = 0; kb < KB; ++kb, dst += kWinGroup * 128) {
          if (tree) {
            tma_load_3d(dst, map_tree, kb * 64, kvh, row, &full[st]);
            if (kBoth) tma_load_3d(dst + Lay::K_BYTES, &p.tm_vt, kb * 64, kvh, row, &full[st]);
          } else {
            tma_load_3d_hint(dst, map_cache, kb * 64, kvh, row, &full[st], stream_policy);
            if (kBoth) tma_load_3d_hint(dst + Lay::K_BYTES, &p.tm_vc, kb * 64, kvh, row, &full[st], stream_policy);
          }
        }
      }
    }
    __syncwarp();
  };
  const bool layout_ok = (smem_u32(sm) & 1023u) == 0;  // 128-byte-swizzled boxes
  if (lane == 0 && rg == 0) {
    for (int i = 0; i < ST; ++i) {
      mbar_init(&full[i], RG);
      mbar_init(&empty[i], RG);
    }
    fence_barrier_init();
  }
  if (kBoth) __syncwarp();
  else __syncthreads();
  if (layout_ok)
    for (int i = 0; i < min(ST, n); ++i) issue(i, i, -1);

  // ---- query rows as B operands, and what each row sees
  __syncthreads();
  uint8_t *s_q = sm + Lay::OFF_Q;
#pragma unroll
  for (int u = tid; u < RB * (D / 8); u += kWinThreads) {
    const int r = u / (D / 8), c = u % (D / 8), row = s_row[r];
    cp_async_16(s_q + (c >> 3) * (RB * 128) + sw128_offset(r, c & 7),
                static_cast<const bf16 *>(p.q) + (size_t)max(row, 0) * D + 8 * c, row >= 0);
  }
  cp_async_commit();
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
  const int lo_last = window_first(L + p.N - 1, p.window);  // no row's window starts later

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
  const uint32_t q_row = (uint32_t)(rg * 8 * NT + (lane & 7)), q_addr = smem_u32(s_q) + q_row * 128u;
  const uint32_t q_chunk = (uint32_t)(lane >> 3);
  auto load_q = [&](int k, uint32_t (&q)[NT][4]) {
    const uint32_t c = 2 * k + q_chunk;
#pragma unroll
    for (int j = 0; j < NT; ++j)
      ldsm_x4(q[j], q_addr + (c >> 3) * (RB * 128) + j * 1024 + (((c & 7) ^ (q_row & 7)) << 4));
  };
  // held for good with one group at a time, loaded for each pair of groups
  constexpr bool kHold = RG == 1 || NT < 4;
  uint32_t held[kHold ? DT / 2 : 1][NT][4];
  if constexpr (kHold) {
#pragma unroll
    for (int k = 0; k < DT; k += 2) load_q(k, held[k / 2]);
  }
  int done = 0, issued = min(ST, n);
  int st = 0, phase = 0;  // the stage of group i and the parity of its use
  // One group at a time, the stage of group i - RG is filled again at the start of group i: two
  // warps that share a slice need not be done with the previous group at the same time.  Two at a
  // time, the stages of the last ones are filled again between the products of the next ones.
  int before = 0;  // groups before i whose stages are not yet filled again
  auto refill = [&](int i) {
    for (; before > 0; --before) {
      if (i - before + ST >= n) continue;
      issue(i - before + ST, st >= before ? st - before : st - before + ST, st >= before ? phase : phase ^ 1);
      ++issued;
    }
  };

  // NG groups from group i on: scores, exponents, weights, outputs.  Two at a time where rows fill
  // the operands (64 of them), so that the matrix instructions of one group hide the operand loads
  // and latencies of the other: 512 units of 64 rows, window 4097, 299 us against 317 one at a
  // time, while 40 rows would take 250 against 233: fewer copies are in flight meanwhile.
  auto work = [&](auto ng, int i) {
    constexpr int NG = decltype(ng)::value;
    uint32_t stage[NG];
#pragma unroll
    for (int g = 0; g < NG; ++g) stage[g] = ring_addr + (st + g >= ST ? st + g - ST : st + g) * Lay::G_BYTES;
    auto load_k = [&](int k, uint32_t (&a)[NG][4]) {
#pragma unroll
      for (int g = 0; g < NG; ++g) ldsm_x4(a[g], stage[g] + (k_off ^ ((k & 3) << 5)) + (k >> 2) * (kWinGroup * 128));
    };
    auto load_v = [&](int d, uint32_t (&a)[NG][4]) {
#pragma unroll
      for (int g = 0; g < NG; ++g)
        ldsm_x4_trans(a[g], stage[g] + Lay::K_BYTES + (v_off ^ ((d & 3) << 5)) + (d >> 2) * (kWinGroup * 128));
    };
    float s[NG][NT][4];
#pragma unroll
    for (int g = 0; g < NG; ++g)
#pragma unroll
      for (int j = 0; j < NT; ++j) s[g][j][0] = s[g][j][1] = s[g][j][2] = s[g][j][3] = 0.f;
    // each step's operands are loaded a step ahead of its products
    uint32_t a[2][NG][4], q[2][NT][4];
    if constexpr (!kHold) load_q(0, q[0]);
    load_k(0, a[0]);
#pragma unroll
    for (int k = 0; k < DT; ++k) {
      if (k + 1 < DT) load_k(k + 1, a[(k + 1) & 1]);
      if (!kHold && k % 2 == 0 && k + 2 < DT) load_q(k + 2, q[(k / 2 + 1) & 1]);
#pragma unroll
      for (int g = 0; g < NG; ++g)
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          const uint32_t *b = kHold ? held[kHold ? k / 2 : 0][j] : q[(k / 2) & 1][j];
          mma_bf16_16816(s[g][j], a[k & 1][g], b[2 * (k & 1)], b[2 * (k & 1) + 1]);
        }
    }
    if (!kHold) refill(i);  // (by now the other warp of the slice is done with those stages too)
#pragma unroll
    for (int g = 0; g < NG; ++g) {
      const int gi = g0 + slice + KS * (i + g);
      const int base = gi < gs ? kWinGroup * (gi < gt ? gi : gi - gt) : first + kWinGroup * (gi - gs);
      // every row sees every key: inside the window of all rows, before the prefix's end
      if (gi >= gs && base >= lo_last && base + kWinGroup <= L) continue;
#pragma unroll
      for (int j = 0; j < NT; ++j) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int r = rg * 8 * NT + 8 * j + 2 * ft + (e & 1), key = base + fg + (e >> 1) * 8;
          bool see;
          if (gi < gt) see = (s_anc[r] >> key) & 1ull;
          else if (gi < gs) see = key < n_sinks;
          else see = key < L && (key >= s_lo[r] || key < p.sinks);
          if (!see) s[g][j][e] = -INFINITY;
        }
      }
      // V rows that no row sees may hold anything: zero them, so that 0 * V stays 0
      const int key = base + k_row;
      const bool live = gi < gt ? key < p.N
                                : (gi < gs ? key < n_sinks : key < L && (key >= lo_root || key < p.sinks));
      if (!live) {
        uint8_t *sv = ring + (stage[g] - ring_addr) + Lay::K_BYTES;
#pragma unroll
        for (int c = 0; c < D / 16; ++c) {
          const int ch = k_chunk * (D / 16) + c;
          *reinterpret_cast<uint4 *>(sv + (ch >> 3) * (kWinGroup * 128) + sw128_offset(k_row, ch & 7)) =
              make_uint4(0, 0, 0, 0);
        }
      }
      fence_proxy_async_smem();  // before the next copy into this stage
      __syncwarp();
    }

    // The weights are taken against a maximum of each row that need not be the latest: only
    // when a score passes it by more than 2^8 (or there is none yet) is it brought up to date
    // over the warp's keys, and the sums and outputs with it.  Then no exchange between
    // lanes is needed but one vote.  (The exponents take the scores' place.)
    float top = -INFINITY;
#pragma unroll
    for (int g = 0; g < NG; ++g)
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) top = fmaxf(top, fmaf(s[g][j][e], sc, -m[j][e & 1]));
    if (__any_sync(0xFFFFFFFFu, top > kWinRescale)) {
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        float w[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float y = fmaxf(s[0][j][e], s[0][j][e + 2]);
          if (NG > 1) y = fmaxf(y, fmaxf(s[NG - 1][j][e], s[NG - 1][j][e + 2]));
          y = fmaxf(y, __shfl_xor_sync(0xFFFFFFFFu, y, 4));
          y = fmaxf(y, __shfl_xor_sync(0xFFFFFFFFu, y, 8));
          y = fmaxf(y, __shfl_xor_sync(0xFFFFFFFFu, y, 16));
          y = fmaxf(y * sc, m[j][e]);
          w[e] = ex2_approx(m[j][e] - y);
          m[j][e] = y;
          l[j][e] *= w[e];
        }
#pragma unroll
        for (int d = 0; d < DT; ++d) {
          o[d][j][0] *= w[0];
          o[d][j][1] *= w[1];
          o[d][j][2] *= w[0];
          o[d][j][3] *= w[1];
        }
      }
    }
    load_v(0, a[0]);
    uint32_t pb[NG][NT][2];
#pragma unroll
    for (int g = 0; g < NG; ++g)
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        float x[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          x[e] = ex2_approx(fmaf(s[g][j][e], sc, -m[j][e & 1]));
          l[j][e & 1] += x[e];
        }
        pb[g][j][0] = transpose_8x8(pack_bf16x2(x[0], x[1]));
        pb[g][j][1] = transpose_8x8(pack_bf16x2(x[2], x[3]));
      }
#pragma unroll
    for (int d = 0; d < DT; ++d) {
      if (d + 1 < DT) load_v(d + 1, a[(d + 1) & 1]);
#pragma unroll
      for (int g = 0; g < NG; ++g)
#pragma unroll
        for (int j = 0; j < NT; ++j) mma_bf16_16816(o[d][j], a[d & 1][g], pb[g][j][0], pb[g][j][1]);
    }
  };
  auto arrived = [&](int at, int par) -> bool {
    return __all_sync(0xFFFFFFFFu, mbar_wait(&full[at], par, abort_flag, p.wait_ns));
  };
  auto step = [&](int count) {  // done with `count` groups
    __syncwarp();               // every lane is
    for (int k = 0; k < count; ++k) {
      if (RG > 1 && lane == 0) mbar_arrive(&empty[st]);
      if (++st == ST) st = 0, phase ^= 1;
    }
    before += count;
  };
  for (int i = 0; layout_ok && i < n;) {
    if constexpr (kHold) {
      if (i >= RG && i - RG + ST < n) {
        issue(i - RG + ST, st >= RG ? st - RG : st - RG + ST, st >= RG ? phase : phase ^ 1);
        ++issued;
      }
    } else if (issued < min(n, i + 2)) {
      refill(i);  // what this step waits for has to be on its way
    }
    if (!arrived(st, phase)) break;
    const int st1 = st + 1 == ST ? 0 : st + 1;
    const bool two = !kHold && i + 1 < n;
    if (two && !arrived(st1, st1 == 0 ? phase ^ 1 : phase)) break;
    done = i + (two ? 2 : 1);
    if constexpr (!kHold) {
      if (two && s_bad[st] == 0 && s_bad[st1] == 0) {
        work(std::integral_constant<int, 2>(), i);
        step(2);
        i += 2;
        continue;
      }
    }
    if (s_bad[st] == 0) work(std::integral_constant<int, 1>(), i);
    step(1);
    ++i;
  }
  if (done < n && layout_ok) {
    // a wait gave up: let the copies in flight land before the shared memory is used again
    *abort_flag = 1;
    const unsigned long long t0 = global_ns();
    for (int i = done; i < issued; ++i)
      while (!mbar_try_wait(&full[i % ST], (i / ST) & 1) && global_ns() - t0 < kWaitLimitNs) {
      }
  }

  // ---- merge the slices: outputs scaled to the CTA's maximum, rows of OS floats
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
  float *acc = reinterpret_cast<float *>(sm);
#pragma unroll
  for (int j = 0; j < NT; ++j)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int r = rg * 8 * NT + 8 * j + 2 * ft + e;
      float top = kWinNone;
#pragma unroll
      for (int k = 0; k < KS; ++k) top = fmaxf(top, s_m[k * RB + r]);
      const float w = ex2_approx(m[j][e] - top);
      float *dst = acc + (size_t)(slice * RB + r) * OS + fg;
#pragma unroll
      for (int d = 0; d < DT; ++d) {
        dst[16 * d] = o[d][j][e] * w;
        dst[16 * d + 8] = o[d][j][e + 2] * w;
      }
    }
  if (tid < RB) {
    float top = kWinNone, sum = 0.f;
#pragma unroll
    for (int k = 0; k < KS; ++k) top = fmaxf(top, s_m[k * RB + tid]);
#pragma unroll
    for (int k = 0; k < KS; ++k) sum += ex2_approx(s_m[k * RB + tid] - top) * s_l[k * RB + tid];
    s_cm[tid] = top;
    s_cl[tid] = sum;
  }
  __syncthreads();
  auto store = [&](int r, int d4, float4 x, float inv) {
    const int row = s_row[r];
    if (row < 0) return;
    *reinterpret_cast<uint2 *>(static_cast<bf16 *>(p.out) + (size_t)row * D + 4 * d4) =
        make_uint2(pack_bf16x2(x.x * inv, x.y * inv), pack_bf16x2(x.z * inv, x.w * inv));
  };
#pragma unroll 4
  for (int u = tid; u < RB * (D / 4); u += kWinThreads) {
    const int r = u / (D / 4), d4 = u % (D / 4);
    float4 x = *reinterpret_cast<const float4 *>(acc + (size_t)r * OS + 4 * d4);
#pragma unroll
    for (int k = 1; k < KS; ++k) {
      const float4 y = *reinterpret_cast<const float4 *>(acc + (size_t)(k * RB + r) * OS + 4 * d4);
      x.x += y.x;
      x.y += y.y;
      x.z += y.z;
      x.w += y.w;
    }
    if (C > 1) *reinterpret_cast<float4 *>(acc + (size_t)r * OS + 4 * d4) = x;
    else store(r, d4, x, s_cl[r] > 0.f ? 1.f / s_cl[r] : 0.f);
  }
  if (C > 1) cluster_merge<D>(acc, OS, s_cm, s_cl, RB, C, rank, kWinNone, store);
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

// 8-column steps of rows per warp, warps per slice and CTAs' worth of rows of a unit: up to four
// steps per warp, two warps per slice beyond 32 rows; more than 64 rows go 64 at a time.
struct WinRows {
  int nt, rg, m_tiles;
};
WinRows window_rows(int M) {
  const int steps = (M + 7) / 8, rg = steps > 4 ? 2 : 1;
  const int nt = rg == 2 ? (steps <= 6 ? 3 : 4) : steps;
  return {nt, rg, (M + 8 * nt * rg - 1) / (8 * nt * rg)};
}

}  // namespace

// The tensor-core kernel pads a unit's rows to 128 or 256 and pays more for a unit's start and
// for the launch, but takes long windows of many rows at twice the rate.  Both sides as fitted
// to measurements (us on 152 SMs, D = 128; 8 to 2048 units, 32 to 512 rows, windows 17 to 4097):
//   here:  10 + units tiles / SMs (3 + 0.28 groups)      (0.2 per group of up to 48 rows)
//   there: 11 + units tiles / SMs (6 + 1.45 key tiles) + 2 SMs / units   (2.55 for 256 rows)
// e.g. 128 units of 104 rows: window 129 16 us against 20, window 1025 43 against 32; 512 units of
// 64 rows: 27 against 39, 82 against 86; 8 units of 208 rows, window 4097: 30 against 85.
// Up to 32 rows this kernel runs at the memory's rate: 2048 units, window 1025: 180 against 270.
bool window_prefers_tc(int B, int N, int Hq, int Hkv, int span, int num_sms) {
  const int M = N * (Hq / Hkv);
  const WinRows r = window_rows(M);
  if (r.rg == 1) return false;
  const double units = (double)B * Hkv, sms = num_sms;
  const double groups = span / kWinGroup + 2 + N / kWinGroup, tiles = span / 128 + 2;
  const double here = 10 + units * r.m_tiles / sms * (3 + (r.nt == 3 ? 0.2 : 0.28) * groups);
  const double there = 11 + units * ((M + 255) / 256) / sms * (6 + (M > 128 ? 2.55 : 1.45) * tiles) + 2 * sms / units;
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
  const WinRows rows_plan = window_rows(a.M);
  const int nt = rows_plan.nt, rg = rows_plan.rg;
  p.m_tiles = rows_plan.m_tiles;
  // CTAs per unit: waves of resident CTAs times the length of one, which costs about 12 groups
  // (its start and merge) beside its share of the window's groups.  (Clusters of 16 gain little on
  // the longest windows and start later: 8 units of 4 rows, window 1024, 7.2 us against 6.6; 16
  // such clusters find no room together, 25 us against 13.)
  const long long units = (long long)a.B * a.Hkv * p.m_tiles, slots = 2ll * num_sms;
  const int span = a.window - 1 < a.cap ? a.window - 1 : a.cap;
  const int groups = span / kWinGroup + (a.N + a.sinks) / kWinGroup + 2;
  long long best = 0;
  p.cluster = 1;
  for (int c = 1; c <= 8; c *= 2) {
    const long long cost = (units * c + slots - 1) / slots * ((groups + c - 1) / c + 12);
    if (c == 1 || cost < best) {
      best = cost;
      p.cluster = c;
    }
  }
  const long long ctas = units * p.cluster;
  if (ctas > INT32_MAX) return cudaErrorInvalidValue;
  return a.D == 128 ? launch_window_d<128>(p, nt, rg, ctas, s) : launch_window_d<64>(p, nt, rg, ctas, s);
}

}  // namespace sv
