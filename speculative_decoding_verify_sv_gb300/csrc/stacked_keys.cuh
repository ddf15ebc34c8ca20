// Listed pages, the own keys behind shared ones, and whole prefixes, for units of few query rows (sm_103a, bf16): the
// kernels are unit_attention.cuh's (a CTA per unit) and warp_units.cuh's (a warp per unit).
//
// Listed pages (sv_sparse_attention): a unit is a sequence, a set of nodes (all of them, or one) and a KV
// head, and its keys are the tree's nodes and the pages of its list, in groups of 16 that none of them
// crosses.  Pages that many rows see together go through the stacked kernel instead, see sparse_plan.
//
// Pieces: the kernel takes the tree's nodes and a sequence's own keys (those behind what it shares; none with
// listed pages), and its rows begin with the stacked kernel's pieces instead of nothing, shared out over the
// slices of the unit's CTAs.  They are read straight to the registers that the products add to, while the first
// keys are on their way.  (One token of 8 requests behind 8192 keys, 19 pieces a row: 19.9 us; without clusters
// 21.9; as one more part of the merge at the end, through shared memory, 25.8; read element by element there,
// 10 us more per CTA.)
#pragma once

#include "unit_attention.cuh"

namespace sv {

struct ListedParams;
struct PieceParams;
struct OwnParams;
// The launches, each in a file of its own; `groups` of 16 keys per unit (for the choice of shapes).
cudaError_t launch_listed_units(ListedParams &p, int D, int groups, int num_sms, cudaStream_t s);
cudaError_t launch_joined_units(PieceParams &p, int D, int num_sms, cudaStream_t s);
cudaError_t launch_own_units(OwnParams &p, int D, int groups, int num_sms, cudaStream_t s);
cudaError_t launch_listed_warps(ListedParams &p, int D, cudaStream_t s);
cudaError_t launch_joined_warps(PieceParams &p, int D, cudaStream_t s);
cudaError_t launch_own_warps(OwnParams &p, int D, cudaStream_t s);

struct ListedParams : WinParams {
  const int32_t *pages;  // [B, sets, Hkv, list_len]
  int list_len, sets, set_nodes, page_size, page_groups;
  int units;  // (a warp each)
};
struct PieceParams : WinParams {
  const int32_t *group_start, *shared_len;  // (NULL: listed pages, no own keys)
  const long long *header;
  const float *part_o;
  const float2 *part_ml;
  int groups, grid, tile_tokens, row_tiles, list_tiles;
  int units;  // (a warp each)
};

struct OwnParams : WinParams {
  const int32_t *group_start, *shared_len;
  int groups;
  int units;  // (a warp each)
};

namespace {

template <int D, int NT, int RG>
__global__ void __launch_bounds__(kWinThreads, 2) own_attn_kernel(const __grid_constant__ OwnParams p);
template <int D, int NT, int RG>
__global__ void __launch_bounds__(kWinThreads, 2) listed_attn_kernel(const __grid_constant__ ListedParams p);
template <int D, int NT, int RG>
__global__ void __launch_bounds__(kWinThreads, 2) joined_attn_kernel(const __grid_constant__ PieceParams p);

struct ListedKeys {
  using Params = ListedParams;
  static constexpr bool kWindow = false, kListed = true, kPieces = false;
  __device__ static __forceinline__ void begin(const Params &) { wait_previous(); }
  __device__ static __forceinline__ int sequence(const Params &p, int bs) { return bs / p.sets; }
  __device__ static __forceinline__ int first_node(const Params &p, int bs) { return bs % p.sets * p.set_nodes; }
  __device__ static __forceinline__ SharedPart shared_part(const Params &, int, bool, SharedPart *) {
    __syncthreads();
    return {};
  }
  __device__ static __forceinline__ SharedPart shared_part_warp(const Params &, int, bool) { return {}; }
  template <int D, int NT, int RG>
  static auto kernel() {
    return listed_attn_kernel<D, NT, RG>;
  }
};

struct JoinedKeys {
  using Params = PieceParams;
  static constexpr bool kWindow = false, kListed = false, kPieces = true;
  // The stacked kernel lets this one be set up when it has itself waited for everything before it, so that
  // only what it writes has to be waited for: the first own keys are on their way before (wait_pieces).
  __device__ static __forceinline__ void begin(const Params &) {}
  __device__ static __forceinline__ int sequence(const Params &, int bs) { return bs; }
  __device__ static __forceinline__ int first_node(const Params &, int) { return 0; }
  // Listed pages: no own keys, and the same work for every list.
  __device__ static __forceinline__ SharedPart listed_part(const Params &p, int b) {
    const int units = p.Hkv * p.row_tiles;
    return {b, INT32_MAX, p.row_tiles, -1, p.list_tiles, b * units, (long long)b * units * p.list_tiles, (long long)p.B * units * p.list_tiles};
  }
  static __device__ __forceinline__ SharedPart none() { return {0, 0, 0, -1, 0, 0, 0, 0}; }
  // Group g; *bad if it does not ascend.  True if it holds sequence b.
  __device__ static __forceinline__ bool group_part(const Params &p, int g, int b, SharedPart *part, int *bad) {
    const int a = p.group_start[g], e = p.group_start[g + 1], len = p.shared_len[g];
    *bad |= a < 0 || e < a || e > p.B;
    *part = none();
    part->start = a;
    part->len = len;
    part->per = (int)(((long long)(e - a) * p.N + 2 * p.tile_tokens - 1) / (2 * p.tile_tokens));
    part->group = g;
    return a <= b && b < e;
  }
  // Waits for the stacked kernel; then the group's share of its work.
  __device__ static __forceinline__ void wait_pieces(const Params &p, SharedPart &part) {
    wait_previous();
    if (part.group < 0) return;
    part.first = p.header[1 + 2 * part.group];
    const long long at = p.header[2 + 2 * part.group];
    part.tiles = (int)(at >> 32);
    part.unit = (int)at;
    part.total = p.header[0];
  }
  __device__ static __forceinline__ SharedPart checked(const Params &p, int b, bool reports, SharedPart part) {
    // (a group's shared keys are every member's)
    if (reports && part.len > p.prefix_len[b]) set_status(p.status, SV_DEV_BAD_PREFIX);
    part.len = min(max(part.len, 0), p.cap) & ~15;
    return part;
  }
  // The group of sequence b, for a CTA and for a warp.  A call with a group_start that does not ascend
  // shares nothing.
  __device__ static __forceinline__ SharedPart shared_part(const Params &p, int b, bool reports, SharedPart *s_part) {
    if (!p.group_start) {
      __syncthreads();
      return listed_part(p, b);
    }
    int bad = 0, found = 0;
    SharedPart part;
    for (int g = threadIdx.x; g < p.groups; g += kWinThreads)
      if (group_part(p, g, b, &part, &bad)) {
        *s_part = part;
        found = 1;
      }
    bad = __syncthreads_or(bad);
    found = __syncthreads_or(found);
    if (bad || !found) return none();
    return checked(p, b, reports && threadIdx.x == 0, *s_part);
  }
  __device__ static __forceinline__ SharedPart shared_part_warp(const Params &p, int b, bool reports) {
    if (!p.group_start) return listed_part(p, b);
    const int lane = threadIdx.x & 31;
    int bad = 0;
    SharedPart mine = none(), part;
    bool found = false;
    for (int g = lane; g < p.groups; g += 32)
      if (group_part(p, g, b, &part, &bad)) {
        mine = part;
        found = true;
      }
    const unsigned who = __ballot_sync(0xFFFFFFFFu, found);
    if (__any_sync(0xFFFFFFFFu, bad) || who == 0) return none();
    const int from = __ffs((int)who) - 1;
    auto share = [&](auto v) { return __shfl_sync(0xFFFFFFFFu, v, from); };
    part = none();
    part.start = share(mine.start);
    part.len = share(mine.len);
    part.per = share(mine.per);
    part.group = share(mine.group);
    return checked(p, b, reports && lane == 0, part);
  }
  // Where the stacked kernel has left the pieces of a row: its unit's share of the work, cut where a
  // CTA's share ends (of C CTAs CTA c has the work items [W c / C, W (c + 1) / C)).
  __device__ static __forceinline__ Pieces pieces_of(const Params &p, int b, int head, int node, int g, const SharedPart &part) {
    Pieces out;
    if (part.tiles == 0) return out;
    const int token = (b - part.start) * p.N + node, tile = token / (2 * p.tile_tokens), in = token % (2 * p.tile_tokens);
    const int unit = head * part.per + tile;  // of the group
    const long long first = part.first + (long long)unit * part.tiles, ctas = min((long long)p.grid, part.total);
    auto cta_of = [&](long long item) {
      const long long x = (item + 1) * ctas - 1;
      return part.total * ctas <= UINT32_MAX ? (int)((unsigned)x / (unsigned)part.total) : (int)(x / part.total);
    };
    const int c0 = cta_of(first), c1 = cta_of(first + part.tiles - 1);
    out.row = (part.unit + unit + c0) * kStackRows + in / p.tile_tokens * 128 + in % p.tile_tokens * p.G + g;
    out.count = c1 - c0 + 1;
    return out;
  }
  // Piece k of a row, 16 bytes u of its D / 4 (a piece is stored by these, rows side by side).
  template <int D>
  __device__ static __forceinline__ const float4 *piece(const Params &p, int row, int k, int u) {
    return reinterpret_cast<const float4 *>(p.part_o) + ((size_t)(row / kStackRows + k) * (D / 4) + u) * kStackRows + row % kStackRows;
  }
  template <int D, int NT, int RG>
  static auto kernel() {
    return joined_attn_kernel<D, NT, RG>;
  }
};

// Every key a sequence's own; the groups are only checked, by the first warp of each sequence's first unit.
struct OwnKeys {
  using Params = OwnParams;
  static constexpr bool kWindow = false, kListed = false, kPieces = false;
  __device__ static __forceinline__ void begin(const Params &) { wait_previous(); }
  __device__ static __forceinline__ int sequence(const Params &, int bs) { return bs; }
  __device__ static __forceinline__ int first_node(const Params &, int) { return 0; }
  __device__ static __forceinline__ SharedPart shared_part_warp(const Params &p, int b, bool reports) {
    if (reports) report_groups(p.group_start, p.shared_len, p.groups, p.B, p.cap, b, p.prefix_len[b], p.status);
    return {};
  }
  __device__ static __forceinline__ SharedPart shared_part(const Params &p, int b, bool reports, SharedPart *) {
    if (threadIdx.x < 32) shared_part_warp(p, b, reports);
    __syncthreads();
    return {};
  }
  template <int D, int NT, int RG>
  static auto kernel() {
    return own_attn_kernel<D, NT, RG>;
  }
};

template <int D, int NT, int RG>
__global__ void __launch_bounds__(kWinThreads, 2) own_attn_kernel(const __grid_constant__ OwnParams p) {
  unit_attention<D, NT, RG, OwnKeys>(p);
}
template <int D, int NT, int RG>
__global__ void __launch_bounds__(kWinThreads, 2) listed_attn_kernel(const __grid_constant__ ListedParams p) {
  unit_attention<D, NT, RG, ListedKeys>(p);
}
template <int D, int NT, int RG>
__global__ void __launch_bounds__(kWinThreads, 2) joined_attn_kernel(const __grid_constant__ PieceParams p) {
  unit_attention<D, NT, RG, JoinedKeys>(p);
}

}  // namespace

}  // namespace sv
