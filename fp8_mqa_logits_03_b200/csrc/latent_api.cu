// latent_api.cu -- the C ABI of the latent cache store and the latent
// attention (include/fp8idx.h): argument checks, schedule plans and launches.
// Host code only.
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdint>
#include <cstring>

#include "../../include/fp8idx.h"
#include "api_common.h"
#include "kernels.cuh"
#include "latent.cuh"

namespace {

using namespace fp8idx;

// The SM count of the current device, asked for once per device.
int sms_cached() {
  static std::atomic<int> of[64];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 0;
  if (dev < 0 || dev >= 64) return device_sms();
  int n = of[dev].load(std::memory_order_relaxed);
  if (n <= 0) of[dev].store(n = device_sms(), std::memory_order_relaxed);
  return n;
}

struct AttnPlan {
  int ncg = 1, parts = 1;
  int min_tiles = 1;
  bool whole_groups = false;
  size_t off_meta = 0, off_group = 0, off_ml = 0, off_o = 0, total = 0;
};

// The workspace's parts, for a grid of `grid` CTAs.
void lay_out(AttnPlan& pl, int64_t grid) {
  int64_t off = kStatusBytes;
  pl.off_meta = off;
  off += round_up(grid * 16, 256);
  pl.off_group = off;
  off += round_up(kSpreadGroups * static_cast<int64_t>(pl.ncg) * 8, 256);
  pl.off_ml = off;
  off += round_up(grid * 2 * kAttnCols * 8, 256);
  pl.off_o = off;
  if (!pl.whole_groups) off += grid * 2 * kAttnCols * kLatent * 4;
  pl.total = static_cast<size_t>(off);
}

// What joining cut groups costs, in tiles of a CTA's time: more where a piece
// has many columns and a group that is cut lies on CTAs that hold others' pieces
// too.  (64 columns, 2048 slots, 120 rows: 66.5 us cut, 62.7 whole, six tiles
// longer; 512 slots, 160 rows: 37.4 and 38.2, fp8 41.1 and 45.4, seven longer;
// 16 columns, 120 rows: 56.9 and 58.3.)
constexpr int64_t kJoinTiles = 4, kJoinTilesWide = 6;

// One CTA per SM, split into column blocks of 64 (a block of every range runs
// at the same time as the others of that range, so that they share its keys
// in L2) and as many ranges of the tile axis as fit; a range holds at least
// min_tiles tiles (two for more than 32 columns, else one), where there are more
// tiles than groups.  Where all groups have the same number of tiles (`uniform`):
//  - the ranges end with groups, so that nothing is left to be joined, if that
//    makes the longest one at most kJoinTiles tiles longer than an even share
//    (kJoinTilesWide for more than 32 columns and fewer than two ranges a group);
//  - or else, if there are no more groups than ranges, every group gets ranges of
//    its own, if that makes the longest one at most kJoinTiles longer.
AttnPlan plan_attn(int64_t groups, int64_t cols, int64_t tiles_per_group, bool uniform, int sms) {
  AttnPlan pl;
  pl.ncg = static_cast<int>(ceil_div(cols, kAttnCols));
  const int64_t nt = std::max<int64_t>(1, tiles_per_group);
  const int64_t tiles = std::max<int64_t>(1, groups * nt);
  // a cut range leaves cols x 2 KB of sums: with many columns as much as some tiles
  pl.min_tiles = cols > 32 ? 2 : 1;
  const int64_t slots = std::max<int64_t>(1, std::min<int64_t>(sms / pl.ncg, kAttnMaxParts));
  // (and a CTA for each group while there are any: two short groups one behind
  // the other take longer than a cut one; 7 x 3 rows of 1 key 19.3 -> 13 us)
  pl.parts = static_cast<int>(std::min<int64_t>(slots, std::max(groups, ceil_div(tiles, pl.min_tiles))));
  if (uniform && groups > 0) {
    const int64_t even = ceil_div(tiles, pl.parts), most = std::min<int64_t>(pl.parts, groups);
    const int64_t each = ceil_div(groups, most), split = std::max<int64_t>(1, pl.parts / groups);
    if (each * nt <= even + (cols > 32 && split == 1 ? kJoinTilesWide : kJoinTiles)) {
      pl.whole_groups = true;
      pl.parts = static_cast<int>(ceil_div(groups, each));
    } else if (groups <= pl.parts && ceil_div(nt, split) <= even + kJoinTiles) {
      pl.parts = static_cast<int>(groups * split);  // a group's own ranges: none holds parts of two
    }
  }
  lay_out(pl, static_cast<int64_t>(pl.parts) * pl.ncg);
  return pl;
}

// What the workspace queries give: enough for these sizes and for all smaller
// ones, though fewer rows may take more (a plan without cut groups has no
// partial sums, and the number of column blocks decides how many CTAs fit).
// The grid is at most one CTA an SM, and a CTA for each tile and column block.
size_t attn_workspace(int64_t groups, int64_t cols, int64_t tiles_per_group, int sms) {
  AttnPlan pl;
  pl.ncg = static_cast<int>(ceil_div(cols, kAttnCols));
  const int64_t tiles = std::max<int64_t>(1, groups) * std::max<int64_t>(1, tiles_per_group);
  lay_out(pl, std::min<int64_t>(std::max(sms, pl.ncg), tiles * pl.ncg));
  return pl.total;
}

int check_latent_shape(int H, int latent, int rope) {
  if (latent != kLatent || rope != kRope)
    return fail(FP8IDX_EUNSUPPORTED, "only 512 latent and 64 rotated values are supported (got %d, %d)", latent, rope);
  if (H < 1 || H > kAttnMaxHeads)
    return fail(FP8IDX_EUNSUPPORTED, "heads must be in [1, %d] (got %d)", kAttnMaxHeads, H);
  return FP8IDX_OK;
}

// The pool: fp8 codes with scales and rotated parts, or bf16 rows alone.
int check_pool(const void* kv, const float* s, const uint16_t* pe, int64_t num_slots) {
  if (num_slots < 0 || num_slots >= (int64_t(1) << 31)) return fail(FP8IDX_EINVAL, "bad pool size");
  if ((s == nullptr) != (pe == nullptr))
    return fail(FP8IDX_EINVAL, "an fp8 pool has both scales and rotated parts, a bf16 pool neither");
  if (num_slots > 0 && !kv) return fail(FP8IDX_EINVAL, "null pool");
  if (!aligned(kv, 16) || !aligned(pe, 16) || !aligned(s, 4))
    return fail(FP8IDX_EINVAL, "pool rows must be 16-byte aligned, scales 4-byte aligned");
  return FP8IDX_OK;
}

int check_strides(const char* what, const void* ptr, int64_t a, int64_t b) {
  if (!aligned(ptr, 16) || a % 8 || b % 8 || a < 0 || b < 0)
    return fail(FP8IDX_EINVAL, "%s must be 16-byte aligned with strides of whole 16 bytes", what);
  return FP8IDX_OK;
}

int check_scale(float scale) {
  if (!(scale > 0.f) || !std::isfinite(scale)) return fail(FP8IDX_EINVAL, "scale must be positive and finite");
  return FP8IDX_OK;
}

int run_attn(LatentAttnParams& p, const AttnPlan& pl, bool paged, bool fp8, void* ws, size_t ws_bytes, float scale,
             void* stream) {
  if (!ws || !aligned(ws, 256)) return fail(FP8IDX_EINVAL, "workspace must be non-null and 256-byte aligned");
  if (ws_bytes < pl.total)
    return fail(FP8IDX_EWORKSPACE, "workspace too small (%zu < %zu bytes)", ws_bytes, pl.total);
  uint8_t* wsb = static_cast<uint8_t*>(ws);
  p.scale_log2 = static_cast<float>(static_cast<double>(scale) * 1.4426950408889634074);
  p.ncg = pl.ncg;
  p.parts = pl.parts;
  p.min_tiles = pl.min_tiles;
  p.whole_groups = pl.whole_groups ? 1 : 0;
  p.group_meta = reinterpret_cast<int2*>(wsb + pl.off_group);
  p.status = reinterpret_cast<int*>(wsb);
  p.meta = reinterpret_cast<int4*>(wsb + pl.off_meta);
  p.part_ml = reinterpret_cast<float2*>(wsb + pl.off_ml);
  p.part_o = reinterpret_cast<float*>(wsb + pl.off_o);
  p.wait_limit_ns = g_wait_limit_ns;
  p.debug_withhold_first_tile = g_debug_withhold;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e = launch_latent_attn(p, fp8, paged, st);
  if (e != cudaSuccess) return cuda_fail(e, "latent attention launch");
  return ok();
}

int64_t topk_tiles(int topk) { return ceil_div(topk, kAttnKeys); }

// Sizes (not negative) whose products below, in int, int64 or bytes, cannot
// overflow: the rows are bounded before anything is multiplied by them.
bool sparse_sizes_fit(int64_t rows, int topk) {
  return rows <= (int64_t(1) << 25) && topk <= (1 << 24) && rows * (topk_tiles(topk) + 1) < (int64_t(1) << 31);
}
bool paged_sizes_fit(int64_t B, int R, int max_blocks) {
  return B <= (int64_t(1) << 25) / R && B * max_blocks < (int64_t(1) << 31) &&
         static_cast<int64_t>(max_blocks) * kPageSize < (int64_t(1) << 31) - kAttnKeys;
}

}  // namespace

extern "C" {

int fp8idx_latent_store(const uint16_t* c, int64_t c_stride, const uint16_t* k_pe, int64_t k_pe_stride, int64_t T,
                        const int64_t* positions, const float* cos_sin, int64_t max_pos, int interleaved,
                        const int64_t* slot, int64_t num_slots, void* kv_pool, float* s_pool, uint16_t* pe_pool,
                        const uint16_t* q_pe, int64_t q_row_stride, int64_t q_head_stride, uint16_t* q_out,
                        int64_t out_row_stride, int64_t out_head_stride, int H, void* stream) {
  if (T < 0 || max_pos < 0) return fail(FP8IDX_EINVAL, "negative size");
  if (T > (int64_t(1) << 32)) return fail(FP8IDX_EINVAL, "T=%lld is too large", (long long)T);
  FP8IDX_TRY(check_pool(kv_pool, s_pool, pe_pool, num_slots));
  if ((q_pe == nullptr) != (q_out == nullptr)) return fail(FP8IDX_EINVAL, "q_pe and q_out go together");
  if (q_pe && (H < 1 || H > kAttnMaxHeads))
    return fail(FP8IDX_EUNSUPPORTED, "heads must be in [1, %d] (got %d)", kAttnMaxHeads, H);
  if (T == 0) return ok();
  if (!c || !k_pe || !positions || !cos_sin || !slot) return fail(FP8IDX_EINVAL, "null pointer");
  FP8IDX_TRY(check_strides("c", c, c_stride, 0));
  FP8IDX_TRY(check_strides("k_pe", k_pe, k_pe_stride, 0));
  if (q_pe) {
    FP8IDX_TRY(check_strides("q_pe", q_pe, q_row_stride, q_head_stride));
    FP8IDX_TRY(check_strides("q_out", q_out, out_row_stride, out_head_stride));
    // the written rows lie apart, whichever of the two strides is the larger
    const bool row_outer = out_row_stride >= out_head_stride;
    const int64_t inner = row_outer ? out_head_stride : out_row_stride, outer = row_outer ? out_row_stride : out_head_stride;
    const int64_t ni = row_outer ? H : T, no = row_outer ? T : H;
    if ((ni > 1 && inner < kRope) || (no > 1 && outer < static_cast<__int128>(ni - 1) * inner + kRope))
      return fail(FP8IDX_EINVAL, "the rows of q_out overlap");
  }
  if (!aligned(cos_sin, 16) || !aligned(positions, 8) || !aligned(slot, 8))
    return fail(FP8IDX_EINVAL, "cos_sin must be 16-byte aligned, positions and slot 8-byte aligned");
  LatentStoreParams p;
  memset(&p, 0, sizeof(p));
  p.c = c;
  p.c_ld = c_stride;
  p.k_pe = k_pe;
  p.pe_ld = k_pe_stride;
  p.positions = positions;
  p.cos_sin = cos_sin;
  p.max_pos = max_pos;
  p.slot = slot;
  p.num_slots = num_slots;
  p.T = T;
  if (s_pool) {
    p.codes = static_cast<uint8_t*>(kv_pool);
    p.scales = s_pool;
    p.pe = pe_pool;
  } else {
    p.kv = static_cast<uint16_t*>(kv_pool);
  }
  p.q_pe = q_pe;
  p.q_out = q_out;
  p.q_row = q_row_stride;
  p.q_head = q_head_stride;
  p.o_row = out_row_stride;
  p.o_head = out_head_stride;
  p.H = H;
  cudaError_t e = launch_latent_store(p, interleaved != 0, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "latent_store launch");
  return ok();
}

size_t fp8idx_sparse_latent_attention_workspace(int64_t rows, int H, int topk) {
  if (rows < 0 || H < 1 || H > kAttnMaxHeads || topk < 0 || !sparse_sizes_fit(rows, topk)) return 0;
  const int sms = sms_cached();
  if (sms <= 0) return 0;
  return attn_workspace(rows, H, topk_tiles(topk), sms);
}

int fp8idx_sparse_latent_attention(const uint16_t* q, int64_t q_row_stride, int64_t q_head_stride,
                                   const void* kv_pool, const float* s_pool, const uint16_t* pe_pool,
                                   int64_t num_slots, const int32_t* slots, int64_t ld_slots, int64_t rows, int topk,
                                   int H, int latent, int rope, float scale, uint16_t* out, float* lse, void* ws,
                                   size_t ws_bytes, void* stream) {
  FP8IDX_TRY(check_latent_shape(H, latent, rope));
  FP8IDX_TRY(check_scale(scale));
  if (rows < 0 || topk < 0) return fail(FP8IDX_EINVAL, "negative size");
  if (!sparse_sizes_fit(rows, topk)) return fail(FP8IDX_EINVAL, "size too large");
  FP8IDX_TRY(check_pool(kv_pool, s_pool, pe_pool, num_slots));
  if (rows == 0) return ok();
  if (!q || !out || (topk > 0 && !slots)) return fail(FP8IDX_EINVAL, "null q, slots or out");
  if (ld_slots < topk) return fail(FP8IDX_EINVAL, "ld_slots (%lld) < topk (%d)", (long long)ld_slots, topk);
  FP8IDX_TRY(check_strides("q", q, q_row_stride, q_head_stride));
  if (!aligned(out, 16) || !aligned(slots, 4) || !aligned(lse, 4))
    return fail(FP8IDX_EINVAL, "out must be 16-byte aligned, slots and lse 4-byte aligned");
  const int sms = sms_cached();
  if (sms <= 0) return fail(FP8IDX_ECUDA, "no CUDA device");
  LatentAttnParams p;
  memset(&p, 0, sizeof(p));
  p.q = q;
  p.q_row = q_row_stride;
  p.q_head = q_head_stride;
  p.kv = static_cast<const uint8_t*>(kv_pool);
  p.s = s_pool;
  p.pe = reinterpret_cast<const uint8_t*>(pe_pool);
  p.num_slots = num_slots;
  p.slots = slots;
  p.ld_slots = ld_slots;
  p.topk = topk;
  p.groups = static_cast<int>(rows);
  p.R = 1;
  p.H = H;
  p.out = out;
  p.lse = lse;
  return run_attn(p, plan_attn(rows, H, topk_tiles(topk), true, sms), false, s_pool != nullptr, ws, ws_bytes, scale, stream);
}

size_t fp8idx_paged_latent_attention_workspace(int64_t B, int R, int max_blocks, int H) {
  if (B < 0 || R < 1 || R > 8 || H < 1 || H > kAttnMaxHeads || max_blocks < 1 || !paged_sizes_fit(B, R, max_blocks)) return 0;
  const int sms = sms_cached();
  if (sms <= 0) return 0;
  return attn_workspace(B, static_cast<int64_t>(R) * H, max_blocks, sms);
}

int fp8idx_paged_latent_attention(const uint16_t* q, int64_t q_row_stride, int64_t q_head_stride,
                                  const void* kv_pages, const float* s_pages, const uint16_t* pe_pages,
                                  const int32_t* block_table, const int32_t* seq_lens, int64_t B, int R,
                                  int max_blocks, int64_t num_pages, int page_size, int H, int latent, int rope,
                                  float scale, uint16_t* out, float* lse, void* ws, size_t ws_bytes, void* stream) {
  FP8IDX_TRY(check_latent_shape(H, latent, rope));
  FP8IDX_TRY(check_scale(scale));
  if (page_size != kPageSize) return fail(FP8IDX_EUNSUPPORTED, "page_size must be 64 (got %d)", page_size);
  if (R < 1 || R > 8) return fail(FP8IDX_EUNSUPPORTED, "rows per request must be in [1, 8] (got %d)", R);
  if (B < 0 || num_pages < 0 || max_blocks < 1) return fail(FP8IDX_EINVAL, "bad sizes");
  if (num_pages >= (int64_t(1) << 31) / kPageSize) return fail(FP8IDX_EINVAL, "pool too large");
  if (!paged_sizes_fit(B, R, max_blocks)) return fail(FP8IDX_EINVAL, "size too large");
  FP8IDX_TRY(check_pool(kv_pages, s_pages, pe_pages, num_pages * kPageSize));
  if (B == 0) return ok();
  if (!q || !out || !block_table || !seq_lens) return fail(FP8IDX_EINVAL, "null q, block_table, seq_lens or out");
  FP8IDX_TRY(check_strides("q", q, q_row_stride, q_head_stride));
  if (!aligned(out, 16) || !aligned(block_table, 4) || !aligned(seq_lens, 4) || !aligned(lse, 4))
    return fail(FP8IDX_EINVAL, "out must be 16-byte aligned, block_table, seq_lens and lse 4-byte aligned");
  const int sms = sms_cached();
  if (sms <= 0) return fail(FP8IDX_ECUDA, "no CUDA device");
  LatentAttnParams p;
  memset(&p, 0, sizeof(p));
  p.q = q;
  p.q_row = q_row_stride;
  p.q_head = q_head_stride;
  p.kv = static_cast<const uint8_t*>(kv_pages);
  p.s = s_pages;
  p.pe = reinterpret_cast<const uint8_t*>(pe_pages);
  p.num_slots = num_pages * kPageSize;
  p.block_table = block_table;
  p.seq_lens = seq_lens;
  p.max_blocks = max_blocks;
  p.groups = static_cast<int>(B);
  p.R = R;
  p.H = H;
  p.out = out;
  p.lse = lse;
  return run_attn(p, plan_attn(B, static_cast<int64_t>(R) * H, max_blocks, false, sms), true, s_pages != nullptr, ws, ws_bytes,
                  scale, stream);
}

}  // extern "C"
