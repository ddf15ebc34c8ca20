// Units of few query rows, a warp each (sm_103a, bf16): many short units.
//
// What unit_attention.cuh does with a CTA per unit, whose four warps share its keys: here each warp takes a
// unit of up to 32 rows alone, with a ring of two groups of 16 keys, and nothing in the kernel waits for
// another warp.  A unit's fixed latencies -- lengths, page ids, the first copies, the end -- then
// overlap with the three other warps' of the CTA and those of the SM's other CTAs, and there is no merge.
// For 2048 units of 20 rows with 264 keys of their own a CTA per unit takes 90 us (11 us each, of which 4
// start, 4 keys, 3 end), a warp per unit 70; few or long units are better off with a CTA (warp_units_pay).
//
// The products and their fragments are those of unit_attention.cuh: S^T = K Q^T, O^T = V^T P^T on
// mma.sync.
#pragma once

#include "unit_attention.cuh"

namespace sv {

namespace {

template <int D, int NT, class Keys>
struct WarpLayout {
  static constexpr int KB = D / 64, RB = 8 * NT;
  static constexpr int K_BYTES = kWinGroup * D * 2, G_BYTES = 2 * K_BYTES;
  static constexpr int ST = 2;
  static constexpr int RING = ST * G_BYTES;
  static constexpr int OFF_Q = 4 * RING;          // [4][RB][D], 128-byte swizzle per 64 columns
  static constexpr int OFF_FULL = OFF_Q + 4 * RB * D * 2;
  static constexpr int OFF_PAR = OFF_FULL + 4 * ST * 8;        // [4][64]
  static constexpr int OFF_ANC = OFF_PAR + 4 * kMaxNodes * 4;  // [4][RB]
  static constexpr int OFF_PIECE = OFF_ANC + 4 * RB * 8;       // [4][RB]
  static constexpr int OFF_ABORT = OFF_PIECE + 4 * RB * 8;
  static constexpr int SMEM = OFF_ABORT + 16;
  static constexpr int CTAS = NT == 1 ? 3 : 2;    // per SM
  static_assert(CTAS * (SMEM + 1024) <= 228 * 1024, "shared memory");
};

template <int D, int NT, class Keys>
__device__ __forceinline__ void warp_units(const typename Keys::Params &p) {
  using Lay = WarpLayout<D, NT, Keys>;
  constexpr int ST = Lay::ST, RB = Lay::RB, DT = D / 16;
  extern __shared__ __align__(1024) uint8_t warp_smem[];
  uint8_t *sm = warp_smem;
  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xFFFFFFFFu, tid >> 5, 0);
  const int fg = lane >> 2, ft = lane & 3;
  uint8_t *ring = sm + warp * Lay::RING, *s_q = sm + Lay::OFF_Q + warp * (RB * D * 2);
  uint64_t *full = reinterpret_cast<uint64_t *>(sm + Lay::OFF_FULL) + warp * ST;
  int *s_par = reinterpret_cast<int *>(sm + Lay::OFF_PAR) + warp * kMaxNodes;
  uint64_t *s_anc = reinterpret_cast<uint64_t *>(sm + Lay::OFF_ANC) + warp * RB;
  Pieces *s_piece = reinterpret_cast<Pieces *>(sm + Lay::OFF_PIECE) + warp * RB;
  volatile int *abort_flag = reinterpret_cast<volatile int *>(sm + Lay::OFF_ABORT);

  const int unit = blockIdx.x * 4 + warp;
  const bool real = unit < p.units;
  const int u = real ? unit : 0, mt = u % p.m_tiles, kvh = u / p.m_tiles % p.Hkv, bs = u / p.m_tiles / p.Hkv;
  const int b = Keys::sequence(p, bs), node0 = Keys::first_node(p, bs);
  const bool reports = real && kvh == 0 && mt == 0 && node0 == 0;
  const bool layout_ok = (smem_u32(sm) & 1023u) == 0;  // 128-byte-swizzled boxes
  if (lane == 0) {
    for (int i = 0; i < ST; ++i) mbar_init(&full[i], 1);
    fence_barrier_init();
  }
  if (tid == 0) *abort_flag = 0;
  // this lane's row: its place in q and out, in heads (-1: past the unit's rows)
  const int R = mt * RB + lane, node = R / p.G, g = R - node * p.G;
  const int my_row = lane < RB && R < p.M ? (b * p.N + node0 + node) * p.Hq + kvh * p.G + g : -1;
  Keys::begin(p);
  int L = p.prefix_len[b], entries = 0;
  if constexpr (Keys::kListed) entries = listed_length(p.pages + ((size_t)bs * p.Hkv + kvh) * p.list_len, p.list_len);
  for (int i = lane; i < kMaxNodes; i += 32) s_par[i] = i < p.N ? tree_parent(p.tree, b, i) : -1;
  // query rows as B operands
#pragma unroll
  for (int i = 0; i < RB * (D / 8) / 32; ++i) {
    const int at = i * 32 + lane, r = at / (D / 8), c = at % (D / 8), row = __shfl_sync(0xFFFFFFFFu, my_row, r);
    cp_async_16(s_q + (c >> 3) * (RB * 128) + sw128_offset(r, c & 7), static_cast<const bf16 *>(p.q) + (size_t)max(row, 0) * D + 8 * c,
                row >= 0);
  }
  cp_async_commit();
  SharedPart shared = Keys::shared_part_warp(p, b, reports);
  if (L < 0 || L > p.cap) {
    if (reports && lane == 0) set_status(p.status, SV_DEV_BAD_PREFIX);
    L = L < 0 ? 0 : p.cap;
  }
  __syncthreads();  // (the abort word)

  // groups: tree nodes, then own keys or listed pages
  const int own = Keys::kPieces ? min(shared.len, L) : 0, first = own & ~(kWinGroup - 1);
  const int gt = (p.N + kWinGroup - 1) / kWinGroup;
  int n = gt;
  if constexpr (Keys::kListed) n += entries * p.page_groups;
  else n += own < L ? (L - first + kWinGroup - 1) / kWinGroup : 0;
  if (!real || !layout_ok) n = 0;
  const uint64_t stream_policy = l2_policy_evict_first(), tree_policy = l2_policy_evict_normal();
  int desc = -1, desc_pos = 0;  // lane i: row and position of group 32 k + i, k the batch being issued
  auto locate = [&](int i) -> int {
    if (i >= n) return -1;
    if (i < gt) {
      desc_pos = kWinGroup * i;
      return b * p.N + kWinGroup * i;
    }
    int page, off;
    if constexpr (Keys::kListed) {
      // group k of the list: 16 keys of one page; a negative entry, and keys past the prefix, are none
      const int k = i - gt;
      page = p.pages[((size_t)bs * p.Hkv + kvh) * p.list_len + k / p.page_groups];
      off = k % p.page_groups * kWinGroup;
      const long long at = (long long)page * p.page_size + off;
      if (page < 0 || at >= L) return -1;
      desc_pos = (int)at;
    } else {
      desc_pos = first + kWinGroup * (i - gt);
      page = p.block_table ? desc_pos / p.block_size : 0;
      off = p.block_table ? desc_pos - page * p.block_size : 0;
    }
    if (!p.block_table) return b * p.Lmax + desc_pos;
    const int blk = p.block_table[(size_t)b * p.max_blocks + page];
    if (blk < 0 || blk >= p.num_blocks) {
      set_status(p.status, SV_DEV_BAD_BLOCK);
      return -1;
    }
    return blk * p.block_size + off;
  };
  int copied = 0;                  // groups issued
  int kept[ST];                    // the group's position in each stage, -1 if it holds no keys
  auto issue = [&](int st) {
    if ((copied & 31) == 0) desc = locate(copied + lane);
    const int row = __shfl_sync(0xFFFFFFFFu, desc, copied & 31), pos = __shfl_sync(0xFFFFFFFFu, desc_pos, copied & 31);
    const bool tree = copied < gt;
    if (elect_one()) {
      if (row < 0) {
        mbar_arrive(&full[st]);
      } else {
        uint8_t *dst = ring + st * Lay::G_BYTES;
        const uint64_t policy = tree ? tree_policy : stream_policy;
        mbar_expect_tx(&full[st], Lay::G_BYTES);
        tma_load_4d_hint(dst, tree ? &p.tm_kt : &p.tm_kc, 0, row, 0, kvh, &full[st], policy);
        tma_load_4d_hint(dst + Lay::K_BYTES, tree ? &p.tm_vt : &p.tm_vc, 0, row, 0, kvh, &full[st], policy);
      }
    }
    __syncwarp();
#pragma unroll
    for (int k = 0; k < ST; ++k)
      if (k == st) kept[k] = row < 0 ? -1 : pos;
    ++copied;
  };
#pragma unroll
  for (int i = 0; i < ST; ++i) {
    kept[i] = -1;
    if (i < n) issue(i);
  }

  if constexpr (Keys::kPieces) Keys::wait_pieces(p, shared);

  // ---- what each row sees of the tree; its pieces
  int count = 0;
  if (lane < RB) {
    uint64_t anc = 0;
    if (my_row >= 0) {
      int depth;
      if (!tree_walk(s_par, node0 + node, &anc, &depth) && kvh == 0) set_status(p.status, SV_DEV_BAD_TREE);
    }
    s_anc[lane] = anc;
    if constexpr (Keys::kPieces) {
      Pieces pieces;
      if (real && my_row >= 0) pieces = Keys::pieces_of(p, b, kvh, node, g, shared);
      s_piece[lane] = pieces;
      count = pieces.count;
    }
  }
  __syncwarp();

  float o[DT][NT][4];
#pragma unroll
  for (int d = 0; d < DT; ++d)
#pragma unroll
    for (int j = 0; j < NT; ++j) o[d][j][0] = o[d][j][1] = o[d][j][2] = o[d][j][3] = 0.f;
  float m[NT][2], l[NT][2];
#pragma unroll
  for (int j = 0; j < NT; ++j) m[j][0] = m[j][1] = kWinNone, l[j][0] = l[j][1] = 0.f;
  if constexpr (Keys::kPieces) {
    // (pieces through shared memory at the end: Medusa trees behind one prompt 143 us instead of 135, 26-node
    // trees over 256 pages 88.5 instead of 81)
    begin_with_pieces<D, NT, Keys>(p, s_piece, count, 0, 1, o, m, l);
  }
  cp_async_wait<0>();
  __syncwarp();
  const float sc = p.scale_log2;
  const int k_row = lane & 15, k_chunk = lane >> 4;
  const int v_row = (lane & 7) + ((lane >> 4) << 3), v_chunk = (lane >> 3) & 1;
  const uint32_t k_off = sw128_offset(k_row, k_chunk), v_off = sw128_offset(v_row, v_chunk);
  const uint32_t ring_addr = smem_u32(ring);
  // query rows, held in registers
  uint32_t held[DT / 2][NT][4];
  {
    const uint32_t q_row = (uint32_t)(lane & 7), q_addr = smem_u32(s_q) + q_row * 128u + ((((uint32_t)lane >> 3) ^ q_row) << 4);
#pragma unroll
    for (int k = 0; k < DT; k += 2)
#pragma unroll
      for (int j = 0; j < NT; ++j) ldsm_x4(held[k / 2][j], (q_addr ^ ((k & 2) << 5)) + (k >> 2) * (RB * 128) + j * 1024);
  }

  int done = 0, st = 0, phase = 0;
  for (int i = 0; i < n; ++i) {
    if (!__all_sync(0xFFFFFFFFu, limited_wait(&full[st], phase, abort_flag, p))) break;
    done = i + 1;
    int pos = -1;
#pragma unroll
    for (int k = 0; k < ST; ++k)
      if (k == st) pos = kept[k];
    if (pos >= 0) {
      const uint32_t stage = ring_addr + st * Lay::G_BYTES;
      float s[NT][4];
      uint32_t a[2][4];
      auto load_k = [&](int k, uint32_t (&x)[4]) { ldsm_x4(x, stage + (k_off ^ ((k & 3) << 5)) + (k >> 2) * (kWinGroup * 128)); };
      load_k(0, a[0]);
#pragma unroll
      for (int k = 0; k < DT; ++k) {
        if (k + 1 < DT) load_k(k + 1, a[(k + 1) & 1]);
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          const uint32_t *q = held[k / 2][j];
          if (k == 0) mma_first(s[j], a[0], q[0], q[1]);
          else mma_bf16_16816(s[j], a[k & 1], q[2 * (k & 1)], q[2 * (k & 1) + 1]);
        }
      }
      const bool tree = i < gt;
      if (tree || pos < own || pos + kWinGroup > L) {
        // what the rows do not see of the group
        const int end = tree ? p.N : L, lo = tree ? 0 : own;
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int key = pos + fg;
            bool see0, see1;
            if (tree) {
              const uint32_t seen = (uint32_t)(s_anc[8 * j + 2 * ft + e] >> pos) >> fg;
              see0 = seen & 1u;
              see1 = seen & 256u;
            } else {
              see0 = key >= lo && key < end;
              see1 = key + 8 >= lo && key + 8 < end;
            }
            if (!see0) s[j][e] = -INFINITY;
            if (!see1) s[j][e + 2] = -INFINITY;
          }
        // V rows that are no keys may hold anything: zero them, so that 0 * V stays 0
        const int key = pos + k_row;
        if (key < lo || key >= end) {
          uint8_t *sv = ring + st * Lay::G_BYTES + Lay::K_BYTES;
#pragma unroll
          for (int c = 0; c < D / 16; ++c) {
            const int ch = k_chunk * (D / 16) + c;
            *reinterpret_cast<uint4 *>(sv + (ch >> 3) * (kWinGroup * 128) + sw128_offset(k_row, ch & 7)) = make_uint4(0, 0, 0, 0);
          }
        }
        fence_proxy_async_smem();  // before the next copy into this stage
        __syncwarp();
      }
      // weights against a maximum that may lag by 2^8
      float x[NT][4], top = -INFINITY;
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          x[j][e] = fmaf(s[j][e], sc, -m[j][e & 1]);
          top = fmaxf(top, x[j][e]);
        }
      if (__any_sync(0xFFFFFFFFu, top > kWinRescale)) {
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
          for (int e = 0; e < 4; ++e) x[j][e] = fmaf(s[j][e], sc, -m[j][e & 1]);
#pragma unroll
          for (int d = 0; d < DT; ++d) {
            o[d][j][0] *= w[0];
            o[d][j][1] *= w[1];
            o[d][j][2] *= w[0];
            o[d][j][3] *= w[1];
          }
        }
      }
      uint32_t pb[NT][2];
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float x0 = ex2_approx(x[j][2 * h]), x1 = ex2_approx(x[j][2 * h + 1]);
          l[j][0] += x0;
          l[j][1] += x1;
          pb[j][h] = transpose_8x8(pack_bf16x2(x0, x1));  // (off by at most 2^-8; the sum is of the unrounded)
        }
      auto load_v = [&](int d, uint32_t (&y)[4]) {
        ldsm_x4_trans(y, stage + Lay::K_BYTES + (v_off ^ ((d & 3) << 5)) + (d >> 2) * (kWinGroup * 128));
      };
      load_v(0, a[0]);
#pragma unroll
      for (int d = 0; d < DT; ++d) {
        if (d + 1 < DT) load_v(d + 1, a[(d + 1) & 1]);
#pragma unroll
        for (int j = 0; j < NT; ++j) mma_bf16_16816(o[d][j], a[d & 1], pb[j][0], pb[j][1]);
      }
    }
    __syncwarp();  // every lane is done with the stage
    if (copied < n) issue(st);
    if (++st == ST) st = 0, phase ^= 1;
  }
  if (done < n) {
    // a wait gave up: let this warp's copies in flight land before the shared memory is given up
    *abort_flag = 1;
    const unsigned long long t0 = global_ns();
    for (int i = done; i < copied; ++i)
      while (!mbar_try_wait(&full[i % ST], (i / ST) & 1) && global_ns() - t0 < kWaitLimitNs) {
      }
    __syncwarp();
  }

  // ---- the end: the rows' sums
#pragma unroll
  for (int j = 0; j < NT; ++j)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      float sum = l[j][e];
      sum += __shfl_xor_sync(0xFFFFFFFFu, sum, 4);
      sum += __shfl_xor_sync(0xFFFFFFFFu, sum, 8);
      sum += __shfl_xor_sync(0xFFFFFFFFu, sum, 16);
      const float inv = sum > 0.f ? 1.f / sum : 0.f;
#pragma unroll
      for (int d = 0; d < DT; ++d) {
        o[d][j][e] *= inv;
        o[d][j][e + 2] *= inv;
      }
    }
  // rows 2 ft and 2 ft + 1 of dimensions fg and fg + 8 become, by a transpose and an exchange of neighbours,
  // four dimensions of row fg
#pragma unroll
  for (int j = 0; j < NT; ++j) {
    const int row = __shfl_sync(0xFFFFFFFFu, my_row, 8 * j + fg);
#pragma unroll
    for (int d = 0; d < DT; ++d) {
      const uint32_t x = transpose_8x8(pack_bf16x2(o[d][j][0], o[d][j][1])), y = transpose_8x8(pack_bf16x2(o[d][j][2], o[d][j][3]));
      const bool odd = lane & 1;
      const uint32_t other = __shfl_xor_sync(0xFFFFFFFFu, odd ? x : y, 1);
      if (real && row >= 0)
        *reinterpret_cast<uint2 *>(static_cast<bf16 *>(p.out) + (size_t)row * D + 16 * d + (odd ? 6 + 2 * ft : 2 * ft)) =
            odd ? make_uint2(other, y) : make_uint2(x, other);
    }
  }
  if (lane == 0) {
    if (!layout_ok) set_status(p.status, SV_DEV_LAYOUT);
    else if (*abort_flag) set_status(p.status, SV_DEV_TIMEOUT);
  }
}

template <int D, int NT, class Keys, class P>
cudaError_t launch_warps_typed(void (*kern)(P), const P &p, cudaStream_t s) {
  constexpr int smem = WarpLayout<D, NT, Keys>::SMEM;
  static std::atomic<bool> attr[64];
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev < 0 || dev >= 64 || !attr[dev].load()) {
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < 64) attr[dev].store(true);
  }
  return launch_close(kern, dim3(((unsigned)p.units + 3) / 4), kWinThreads, (size_t)smem, s, p);
}

// Launches kernel(D, 8-column steps of a unit's rows).
template <class Keys, class P, class K>
cudaError_t launch_warps(const P &p, int D, cudaStream_t s, K kernel) {
  auto of = [&](auto d) {
    constexpr int DD = decltype(d)::value;
    auto step = [&](auto nt) {
      constexpr int NT = decltype(nt)::value;
      return launch_warps_typed<DD, NT, Keys, P>(kernel(d, nt), p, s);
    };
    switch (((p.M + p.m_tiles - 1) / p.m_tiles + 7) / 8) {
      case 1: return step(std::integral_constant<int, 1>());
      case 2: return step(std::integral_constant<int, 2>());
      case 3: return step(std::integral_constant<int, 3>());
      default: return step(std::integral_constant<int, 4>());
    }
  };
  return D == 128 ? of(std::integral_constant<int, 128>()) : of(std::integral_constant<int, 64>());
}

}  // namespace

}  // namespace sv
