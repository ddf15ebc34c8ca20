// Listed pages, and the own keys behind shared ones, for units of few query rows (sm_103a, bf16): the
// kernel is unit_attention.cuh's; plans and launches of sv_shared_attention and sv_sparse_attention.
//
// Listed pages (sv_sparse_attention): a unit is a sequence, a set of nodes (all of them, or one) and a KV
// head, and its keys are the tree's nodes and the pages of its list, in groups of 16 that none of them
// crosses.  Pages that many rows see together go through the stacked kernel instead, see sparse_plan.
//
// Pieces: the kernel takes the tree's nodes and a sequence's own keys (those behind what it shares; none
// with listed pages), and joins the stacked kernel's pieces of the same rows in its merge, as one more part
// beside those of its own warps.  A row's first piece is copied to shared memory while the keys are worked
// on, the others (units that were cut) follow through the ring's room.  (Read straight from memory in the
// merge, element by element, they took 10 us per CTA.)
#include "unit_attention.cuh"

namespace sv {

namespace {

struct ListedParams : WinParams {
  const int32_t *pages;  // [B, sets, Hkv, list_len]
  int list_len, sets, set_nodes, page_size, page_groups;
};
struct PieceParams : WinParams {
  const int32_t *group_start, *shared_len;  // (NULL: listed pages, no own keys)
  const long long *header;
  const float *part_o;
  const float2 *part_ml;
  int groups, grid, tile_tokens, row_tiles, list_tiles;
};

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
  template <int D, int NT, int RG>
  static auto kernel() {
    return listed_attn_kernel<D, NT, RG>;
  }
};

struct JoinedKeys {
  using Params = PieceParams;
  static constexpr bool kWindow = false, kListed = false, kPieces = true;
  __device__ static __forceinline__ void begin(const Params &) { wait_previous(); }
  __device__ static __forceinline__ int sequence(const Params &, int bs) { return bs; }
  __device__ static __forceinline__ int first_node(const Params &, int) { return 0; }
  // The group of sequence b and its share of the stacked kernel's work, in one round trip to memory.  A call
  // with a group_start that does not ascend shares nothing.
  __device__ static __forceinline__ SharedPart shared_part(const Params &p, int b, bool reports, SharedPart *s_part) {
    if (!p.group_start) {  // listed pages: no own keys
      __syncthreads();
      return {b, INT32_MAX, p.list_tiles, p.row_tiles, b * p.Hkv * p.row_tiles, (long long)b * p.Hkv * p.row_tiles * p.list_tiles,
              (long long)p.B * p.Hkv * p.row_tiles * p.list_tiles};
    }
    int bad = 0, found = 0;
    for (int g = threadIdx.x; g < p.groups; g += kWinThreads) {
      const int a = p.group_start[g], e = p.group_start[g + 1], len = p.shared_len[g];
      const long long first = p.header[1 + 2 * g], at = p.header[2 + 2 * g], total = p.header[0];
      bad |= a < 0 || e < a || e > p.B;
      if (a <= b && b < e) {
        const int per = (int)(((long long)(e - a) * p.N + 2 * p.tile_tokens - 1) / (2 * p.tile_tokens));
        *s_part = {a, len, (int)(at >> 32), per, (int)at, first, total};
        found = 1;
      }
    }
    bad = __syncthreads_or(bad);
    found = __syncthreads_or(found);
    if (bad || !found) return {0, 0, 0, 0, 0, 0, 0};
    SharedPart part = *s_part;
    // (a group's shared keys are every member's)
    if (reports && threadIdx.x == 0 && part.len > p.prefix_len[b]) set_status(p.status, SV_DEV_BAD_PREFIX);
    part.len = min(max(part.len, 0), p.cap) & ~15;
    return part;
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

template <int D, int NT, int RG>
__global__ void __launch_bounds__(kWinThreads, 2) listed_attn_kernel(const __grid_constant__ ListedParams p) {
  unit_attention<D, NT, RG, ListedKeys>(p);
}
template <int D, int NT, int RG>
__global__ void __launch_bounds__(kWinThreads, 2) joined_attn_kernel(const __grid_constant__ PieceParams p) {
  unit_attention<D, NT, RG, JoinedKeys>(p);
}

size_t up(size_t x) { return (x + 255) / 256 * 256; }

// The workspace of `pieces` pieces behind `header` bytes.
void place(StackPlan &pl, size_t header, long long pieces, int D) {
  pl.pieces = pieces;
  pl.off_ml = up(header);
  pl.off_o = pl.off_ml + up((size_t)pieces * kStackRows * sizeof(float2));
  pl.ws_bytes = pl.off_o + (size_t)pieces * kStackRows * D * sizeof(float);
}

// The largest power of two that divides a page, up to a key tile: the rows of a copy.
int box_of(int page) {
  const int low = page & -page;
  return low < 128 ? low : 128;
}

cudaError_t launch_stack(StackParams &p, const AttnParams &a, const StackPlan &pl, void *ws, bool listed, int box, cudaStream_t s) {
  const long long rows = a.block_table ? (long long)a.num_blocks * a.block_size : (long long)a.B * (a.Lmax > 0 ? a.Lmax : 1);
  p.box_rows = box;
  p.grouped = a.block_table && a.D == 128 && box < 128 && tma_pages_map(&p.tm_k, a.cache_k, a.Hkv, rows, box) &&
              tma_pages_map(&p.tm_v, a.cache_v, a.Hkv, rows, box);
  if (!p.grouped && (!tma_heads_map(&p.tm_k, a.cache_k, a.D, a.Hkv, rows, 1, box) ||
                     !tma_heads_map(&p.tm_v, a.cache_v, a.D, a.Hkv, rows, 1, box)))
    return cudaErrorInvalidValue;
  if (!tma_heads_map(&p.tm_q, a.q, a.D, a.Hq, (long long)a.B * a.N, a.G, pl.tile_tokens)) return cudaErrorInvalidValue;
  char *w = static_cast<char *>(ws);
  p.header = reinterpret_cast<long long *>(w);
  p.part_ml = reinterpret_cast<float2 *>(w + pl.off_ml);
  p.part_o = reinterpret_cast<float *>(w + pl.off_o);
  p.prefix_len = a.prefix_len;
  p.block_table = a.block_table;
  p.status = a.status;
  p.B = a.B;
  p.N = a.N;
  p.Hkv = a.Hkv;
  p.G = a.G;
  p.tile_tokens = pl.tile_tokens;
  p.row_tiles = pl.row_tiles;
  p.list_tiles = pl.list_tiles;
  p.list_work = (long long)a.B * a.Hkv * pl.row_tiles * pl.list_tiles;
  p.Lmax = a.Lmax;
  p.block_size = a.block_size;
  p.max_blocks = a.max_blocks;
  p.num_blocks = a.num_blocks;
  p.cap = a.cap;
  p.scale_log2 = a.scale_log2;
  p.wait_ns = a.wait_ns;
  return launch_stacked(p, a.D, listed, pl.grid, s);
}

cudaError_t launch_joined(const AttnParams &a, const StackParams &st, const StackPlan &pl, int groups_of_keys, cudaStream_t s) {
  PieceParams p{};
  if (!unit_params(p, a, a.M)) return cudaErrorInvalidValue;
  p.group_start = st.group_start;
  p.shared_len = st.shared_len;
  p.header = st.header;
  p.part_o = st.part_o;
  p.part_ml = st.part_ml;
  p.groups = st.groups;
  p.grid = pl.grid;
  p.tile_tokens = pl.tile_tokens;
  p.row_tiles = pl.row_tiles;
  p.list_tiles = pl.list_tiles;
  return launch_units<JoinedKeys>(p, a.D, (long long)a.B * a.Hkv, groups_of_keys, pl.grid, s);
}

}  // namespace

StackPlan shared_plan(int B, int N, int Hq, int Hkv, int D, int groups, int num_sms) {
  StackPlan pl{};
  pl.grid = num_sms > 0 ? num_sms : 152;
  pl.stacked = true;
  pl.tile_tokens = 128 / (Hq / Hkv);
  const long long units = (((long long)B * N + 2 * pl.tile_tokens - 1) / (2 * pl.tile_tokens) + groups) * Hkv;
  place(pl, (1 + 2 * (size_t)groups) * sizeof(long long), units + pl.grid, D);
  return pl;
}

StackPlan sparse_plan(int B, int N, int Hq, int Hkv, int D, int page_size, int list_len, int sets, int num_sms) {
  StackPlan pl{};
  const int G = Hq / Hkv;
  pl.grid = num_sms > 0 ? num_sms : 152;
  if (sets != 1 || N * G <= 32) return pl;
  pl.stacked = true;
  pl.tile_tokens = 128 / G;
  pl.row_tiles = (N + 2 * pl.tile_tokens - 1) / (2 * pl.tile_tokens);
  pl.list_tiles = (int)(((long long)list_len * page_size + 127) / 128);
  place(pl, 0, (long long)B * Hkv * pl.row_tiles + pl.grid, D);
  return pl;
}

cudaError_t launch_shared_attention(const AttnParams &a, const ListArgs &l, const StackPlan &pl, void *ws, cudaStream_t s,
                                    bool (*fails)(), unsigned *launches) {
  StackParams p{};
  p.group_start = l.group_start;
  p.shared_len = l.shared_len;
  p.groups = l.groups;
  if (fails()) return cudaErrorLaunchFailure;
  cudaError_t e = launch_stack(p, a, pl, ws, false, a.block_table ? box_of(a.block_size) : 128, s);
  if (e != cudaSuccess) return e;
  ++*launches;
  if (fails()) return cudaErrorLaunchFailure;
  e = launch_joined(a, p, pl, a.N / kWinGroup + 18, s);
  if (e == cudaSuccess) ++*launches;
  return e;
}

cudaError_t launch_sparse_attention(const AttnParams &a, const ListArgs &l, const StackPlan &pl, void *ws, int num_sms,
                                    cudaStream_t s, bool (*fails)(), unsigned *launches) {
  cudaError_t e;
  if (fails()) return cudaErrorLaunchFailure;
  if (pl.stacked) {
    StackParams p{};
    p.pages = l.pages;
    p.list_len = l.list_len;
    p.page_size = l.page_size;
    e = launch_stack(p, a, pl, ws, true, box_of(l.page_size), s);
    if (e != cudaSuccess) return e;
    ++*launches;
    if (fails()) return cudaErrorLaunchFailure;
    e = launch_joined(a, p, pl, a.N / kWinGroup + 1, s);
  } else {
    ListedParams p{};
    const int set_nodes = a.N / l.sets;
    if (!unit_params(p, a, set_nodes * a.G)) return cudaErrorInvalidValue;
    p.pages = l.pages;
    p.list_len = l.list_len;
    p.sets = l.sets;
    p.set_nodes = set_nodes;
    p.page_size = l.page_size;
    p.page_groups = l.page_size / kWinGroup;
    e = launch_units<ListedKeys>(p, a.D, (long long)a.B * l.sets * a.Hkv, l.list_len * p.page_groups + a.N / kWinGroup + 1, num_sms, s);
  }
  if (e == cudaSuccess) ++*launches;
  return e;
}

}  // namespace sv
