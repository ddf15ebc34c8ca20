// Plans and launches of sv_shared_attention and sv_sparse_attention (bf16).
#include "stacked_keys.cuh"

namespace sv {

namespace {

// Whether a warp per unit is the better shape: with four units per SM or more, where a CTA per unit comes in
// waves.  Measured on 152 SMs, units of 4 rows (one node, 32:8 heads), us a warp / a CTA per unit:
//   listed pages   304 units of 128 keys 8.2 / 7.0, of 4096 keys 150 / 94;  608 units 9.7 / 13.7, 192 / 182;
//                  1216 units 15.5 / 24, 348 / 354
//   own keys       304 units of 16 keys 15.7 / 15.5, of 512 keys 34 / 24;  608 units 16.8 / 22.5, 40 / 42;
//                  1216 units 18.2 / 35, 60 / 73 (with the shared part, 512 keys, before them)
// Tiles are of up to 32 rows.
template <class P>
bool warp_units_pay(P &p, long long kv_units, int num_sms) {
  const int tiles = (p.M + 31) / 32;
  const long long units = kv_units * tiles;
  if (units < 4ll * num_sms || units > INT32_MAX) return false;
  p.m_tiles = tiles;
  p.units = (int)units;
  return true;
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

cudaError_t launch_joined(const AttnParams &a, const StackParams &st, const StackPlan &pl, cudaStream_t s) {
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
  return warp_units_pay(p, (long long)a.B * a.Hkv, pl.grid) ? launch_joined_warps(p, a.D, s)
                                                                           : launch_joined_units(p, a.D, pl.grid, s);
}

}  // namespace

// Shared prefixes are worth the stacked kernel and its pieces where there is much to read, as far as the host can
// know (the lengths are the device's).  Measured, us stacked / every sequence's own rows, one group, keys of all
// units in thousands:
//   one token, 32:8 heads   4 requests of 4096 keys (133) 18.7 / 9.8;  64 of 256 (172) 19 / 13;  16 of 4096 (534) 19 / 22;
//                           64 of 4096 (2138) 31 / 73
//   8 nodes, 64:8 heads     16 of 1024 (141) 31 / 21;  256 of 32 (229) 90 / 39;  16 of 4096 (534) 40 / 60
//   64 nodes, 32:32 heads   16 of 256 (172) 37 / 31;  64 of 32 (229) 108 / 60;  4 of 4096 (534) 47 / 64
StackPlan shared_plan(int B, int N, int Hq, int Hkv, int D, int max_prefix, int groups, int num_sms) {
  StackPlan pl{};
  pl.grid = num_sms > 0 ? num_sms : 152;
  const double reads = (double)B * Hkv * (((long long)N * (Hq / Hkv) + 63) / 64) * max_prefix;  // keys that units read
  if (reads < 1800. * pl.grid || max_prefix <= 128) return pl;
  pl.stacked = true;
  pl.tile_tokens = 128 / (Hq / Hkv);
  const long long units = (((long long)B * N + 2 * pl.tile_tokens - 1) / (2 * pl.tile_tokens) + groups) * Hkv;
  place(pl, (1 + 2 * (size_t)groups) * sizeof(long long), units + pl.grid, D);
  return pl;
}

// Many rows with one list are worth the stacked kernel, which reads a list's K and V once per 256 rows instead
// of once per 64 or 32 but leaves pieces to a second kernel, where there is much to read.  Measured, us stacked /
// in units, pages of 16, 8 KV heads:
//   104 rows (26 nodes, 4 heads)   16 requests with lists of 256 keys 24 / 16, 1024 keys 37 / 36, 4096 keys 76 / 118;
//                                  64 requests 46 / 49, 85 / 144, 223 / 521;  one request, 4096 keys, 21 / 17
//   512 rows                       one request, 1024 keys, 23 / 17, 4096 keys 29 / 39;  16 requests of 256 keys 49 / 55
//   64 rows                        64 requests of 256 keys 32 / 23, of 2048 keys 118 / 134;  16 of 4096 keys 70 / 64
//   up to 48 rows                  64 requests of 4096 keys 205 / 191 (48 rows), 208 / 155 (20 rows)
StackPlan sparse_plan(int B, int N, int Hq, int Hkv, int D, int page_size, int list_len, int sets, int num_sms) {
  StackPlan pl{};
  const int G = Hq / Hkv;
  pl.grid = num_sms > 0 ? num_sms : 152;
  const double reads = (double)B * Hkv * ((N * G + 63) / 64) * list_len * page_size;  // keys that units read
  if (sets != 1 || N * G <= 48 || reads < (N * G > 64 ? 1800. : 4000.) * pl.grid) return pl;
  pl.stacked = true;
  pl.tile_tokens = 128 / G;
  pl.row_tiles = (N + 2 * pl.tile_tokens - 1) / (2 * pl.tile_tokens);
  pl.list_tiles = (int)(((long long)list_len * page_size + 127) / 128);
  place(pl, 0, (long long)B * Hkv * pl.row_tiles + pl.grid, D);
  return pl;
}

cudaError_t launch_shared_attention(const AttnParams &a, const ListArgs &l, const StackPlan &pl, void *ws, cudaStream_t s,
                                    bool (*fails)(), unsigned *launches) {
  if (fails()) return cudaErrorLaunchFailure;
  if (!pl.stacked) {
    OwnParams o{};
    if (!unit_params(o, a, a.M)) return cudaErrorInvalidValue;
    o.group_start = l.group_start;
    o.shared_len = l.shared_len;
    o.groups = l.groups;
    const cudaError_t e = warp_units_pay(o, (long long)a.B * a.Hkv, pl.grid)
                              ? launch_own_warps(o, a.D, s)
                              : launch_own_units(o, a.D, (a.cap + a.N) / kWinGroup + 2, pl.grid, s);
    if (e == cudaSuccess) ++*launches;
    return e;
  }
  StackParams p{};
  p.group_start = l.group_start;
  p.shared_len = l.shared_len;
  p.groups = l.groups;
  cudaError_t e = launch_stack(p, a, pl, ws, false, a.block_table ? box_of(a.block_size) : 128, s);
  if (e != cudaSuccess) return e;
  ++*launches;
  if (fails()) return cudaErrorLaunchFailure;
  e = launch_joined(a, p, pl, s);
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
    e = launch_joined(a, p, pl, s);
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
    const int groups = l.list_len * p.page_groups + a.N / kWinGroup + 1;
    e = warp_units_pay(p, (long long)a.B * l.sets * a.Hkv, num_sms) ? launch_listed_warps(p, a.D, s)
                                                                            : launch_listed_units(p, a.D, groups, num_sms, s);
  }
  if (e == cudaSuccess) ++*launches;
  return e;
}

}  // namespace sv
