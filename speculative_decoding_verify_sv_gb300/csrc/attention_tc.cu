// Tensor-core tree attention: eligibility, plan, tensor maps and launch; the kernel is
// attention_tc_kernel.cuh, its window instances are compiled in attention_tc_window.cu.
#include <cudaTypedefs.h>

#include "attention_tc_kernel.cuh"

namespace sv {

cudaError_t launch_tc_window(const TcParams &p, int D, const TcPlan &pl, cudaStream_t s);
cudaError_t launch_tc_window_paged(const TcParams &p, int D, const TcPlan &pl, cudaStream_t s);

namespace {

PFN_cuTensorMapEncodeTiled_v12000 encoder() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  if (!fn) {
    cudaDriverEntryPointQueryResult q;
    void *ptr = nullptr;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault,
                                         &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(ptr);
  }
  return fn;
}

// 3-D bf16 view (D, heads, rows) with a (64, box1, box2) box, 128-byte swizzle.
bool map3d(CUtensorMap *m, const void *base, int D, int heads, long long rows, int box1,
           int box2) {
  PFN_cuTensorMapEncodeTiled_v12000 enc = encoder();
  if (!enc) return false;
  cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)heads, (cuuint64_t)rows};
  cuuint64_t strides[2] = {(cuuint64_t)D * 2, (cuuint64_t)D * 2 * heads};
  cuuint32_t box[3] = {64u, (cuuint32_t)box1, (cuuint32_t)box2};
  cuuint32_t es[3] = {1, 1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(base), dims, strides, box,
             es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) ==
         CUDA_SUCCESS;
}

// The pages of a paged cache as a 5-D bf16 view (64 columns, 8 rows, 2 column halves,
// groups of 8 rows, heads) with a (64, 8, 2, page_rows / 8, 1) box, 128-byte swizzle: one
// copy brings both 64-column halves of a page, as page_rows / 8 groups of 2 KB (the grouped
// tile layout).  D = 128 only.  rows must be a multiple of 8.
bool map5d_pages(CUtensorMap *m, const void *base, int heads, long long rows, int page_rows) {
  PFN_cuTensorMapEncodeTiled_v12000 enc = encoder();
  if (!enc || rows % 8 != 0 || page_rows % 8 != 0 || page_rows / 8 > 256) return false;
  const cuuint64_t row_bytes = (cuuint64_t)128 * 2 * heads;  // one position, all heads
  cuuint64_t dims[5] = {64, 8, 2, (cuuint64_t)(rows / 8), (cuuint64_t)heads};
  cuuint64_t strides[4] = {row_bytes, 128, 8 * row_bytes, 256};
  cuuint32_t box[5] = {64u, 8u, 2u, (cuuint32_t)(page_rows / 8), 1u};
  cuuint32_t es[5] = {1, 1, 1, 1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 5, const_cast<void *>(base), dims, strides, box,
             es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) ==
         CUDA_SUCCESS;
}

}  // namespace

// 4-D bf16 view (64 columns, rows, column blocks, heads) with a (64, box_rows, D / 64, 1) box,
// 128-byte swizzle: one copy brings box_rows rows of a head, a 64-column block after the other.
bool tma_rows_map(CUtensorMap *m, const void *base, int D, int heads, long long rows, int box_rows) {
  PFN_cuTensorMapEncodeTiled_v12000 enc = encoder();
  if (!enc) return false;
  cuuint64_t dims[4] = {64, (cuuint64_t)rows, (cuuint64_t)(D / 64), (cuuint64_t)heads};
  cuuint64_t strides[3] = {(cuuint64_t)D * 2 * heads, 128, (cuuint64_t)D * 2};
  cuuint32_t box[4] = {64u, (cuuint32_t)box_rows, (cuuint32_t)(D / 64), 1u};
  cuuint32_t es[4] = {1, 1, 1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void *>(base), dims, strides, box, es,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool tc_eligible(sv_dtype dt, int N, int Hq, int Hkv, int D, int paged_block_size) {
  if (dt != SV_BF16 || (D != 64 && D != 128) || N > 64 || Hkv < 1 || Hq % Hkv != 0) return false;
  const int G = Hq / Hkv;
  if (G < 1 || G > 128 || 128 % G != 0) return false;
  if (paged_block_size > 0) {
    // a tile's rows must be whole pages or whole 128-row spans of a page
    const int bs = paged_block_size;
    if (!(bs == 16 || bs == 32 || bs == 64 || (bs >= 128 && bs % 128 == 0))) return false;
  }
  return encoder() != nullptr;
}

TcPlan tc_plan(int B, int N, int Hq, int Hkv, int D, int num_sms) {
  TcPlan pl{};
  const int G = Hq / Hkv;
  const int M = N * G;
  pl.MT = M > kRows ? 2 : 1;
  // row copies spread a small M over all four TMEM lane quarters (see the kernel)
  pl.CP = 1;
  if (pl.MT == 1 && M <= 32 && 32 % G == 0) pl.CP = 4;
  else if (pl.MT == 1 && M <= 64 && 64 % G == 0) pl.CP = 2;
  pl.BN = 128;  // keys per tile
  pl.m_groups = (M + pl.MT * kRows - 1) / (pl.MT * kRows);
  pl.grid = num_sms > 0 ? num_sms : 152;
  const long long units = (long long)B * Hkv * pl.m_groups;
  const long long slots = units + pl.grid;
  const int rows = pl.MT * kRows;
  auto up = [](size_t x) { return (x + 255) / 256 * 256; };
  pl.off_hdr = 0;
  pl.off_flags = 256;
  pl.off_ml = pl.off_flags + up((size_t)slots * 8);
  pl.off_o = pl.off_ml + up((size_t)slots * rows * 2 * 4);
  pl.ws_bytes = pl.off_o + up((size_t)slots * rows * D * 4);
  return pl;
}

cudaError_t launch_attention_tc(const AttnParams &a, const TcPlan &pl, void *ws, cudaStream_t s) {
  TcParams p{};
  const int G = a.G;
  const int rows_q = pl.MT * kRows / pl.CP;  // query rows per TMA box (one row copy)
  const int BN = pl.BN;
  const bool win = a.window > 0;
  const int tree_box = win ? SV_MAX_TREE_NODES : BN;  // rows of a tree tile's box
  if (!map3d(&p.tm_q, a.q, a.D, a.Hq, (long long)a.B * a.N, G, rows_q / G) ||
      !map3d(&p.tm_kt, a.k_tree, a.D, a.Hkv, (long long)a.B * a.N, 1, tree_box) ||
      !map3d(&p.tm_vt, a.v_tree, a.D, a.Hkv, (long long)a.B * a.N, 1, tree_box))
    return cudaErrorInvalidValue;
  if (a.block_table == nullptr) {
    const long long rows = (long long)a.B * (a.Lmax > 0 ? a.Lmax : 1);
    if (!map3d(&p.tm_kc, a.cache_k, a.D, a.Hkv, rows, 1, BN) ||
        !map3d(&p.tm_vc, a.cache_v, a.D, a.Hkv, rows, 1, BN))
      return cudaErrorInvalidValue;
    p.paged = 0;
    p.page_rows = BN;
  } else {
    p.page_rows = a.block_size < BN ? a.block_size : BN;
    const long long rows = (long long)a.num_blocks * a.block_size;
    if (!map3d(&p.tm_kc, a.cache_k, a.D, a.Hkv, rows, 1, p.page_rows) ||
        !map3d(&p.tm_vc, a.cache_v, a.D, a.Hkv, rows, 1, p.page_rows))
      return cudaErrorInvalidValue;
    p.paged = 1;
    // pages shorter than a tile: one copy per page (both column halves) instead of two,
    // into the grouped layout; the plain layout stays when the 5-D view is not available
    p.pg_grouped = a.D == 128 && p.page_rows < BN &&
                   map5d_pages(&p.tm_kc5, a.cache_k, a.Hkv, rows, p.page_rows) &&
                   map5d_pages(&p.tm_vc5, a.cache_v, a.Hkv, rows, p.page_rows);
  }
  if (win) {
    const long long rows = a.block_table ? (long long)a.num_blocks * a.block_size : (long long)a.B * (a.Lmax > 0 ? a.Lmax : 1);
    if (!map3d(&p.tm_ks, a.cache_k, a.D, a.Hkv, rows, 1, 16) || !map3d(&p.tm_vs, a.cache_v, a.D, a.Hkv, rows, 1, 16))
      return cudaErrorInvalidValue;
    p.window = a.window;
    p.sinks = a.sinks;
    // a paged tile starts with a page (or, in longer pages, at a multiple of the tile)
    p.win_align = a.block_table ? p.page_rows : 1;
    p.block_shift = -1;
    for (int k = 4; k < 31; ++k)
      if (a.block_size == 1 << k) p.block_shift = k;
  }
  uint8_t *w = static_cast<uint8_t *>(ws);
  p.hdr = reinterpret_cast<unsigned long long *>(w + pl.off_hdr);
  p.flags = reinterpret_cast<unsigned long long *>(w + pl.off_flags);
  p.part_ml = reinterpret_cast<float *>(w + pl.off_ml);
  p.part_o = reinterpret_cast<float *>(w + pl.off_o);
  p.prefix_len = a.prefix_len;
  p.block_table = a.block_table;
  p.out = a.out;
  p.status = a.status;
  p.B = a.B;
  p.N = a.N;
  p.Hq = a.Hq;
  p.Hkv = a.Hkv;
  p.G = G;
  p.M = a.N * G;
  p.m_groups = pl.m_groups;
  p.upb = a.Hkv * pl.m_groups;
  p.bn = BN;
  p.vt = (long long)a.B * p.upb <= 2LL * pl.grid ? kUnitStartSlots : 0;
  p.Lmax = a.Lmax;
  p.block_size = a.block_size;
  p.max_blocks = a.max_blocks;
  p.num_blocks = a.num_blocks;
  p.cap = a.cap;
  p.scale_log2 = a.scale_log2;
  p.tree = a.tree;
  p.wait_ns = a.wait_ns;
  if (!win) return launch_tc_plan<false, false>(p, a.D, pl, s);
  return p.paged ? launch_tc_window_paged(p, a.D, pl, s) : launch_tc_window(p, a.D, pl, s);
}

}  // namespace sv
