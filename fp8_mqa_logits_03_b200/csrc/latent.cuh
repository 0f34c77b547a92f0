// latent.cuh -- parameter blocks and launch helpers of the latent-attention
// kernels (the cache store, and attention over selected or over all cached
// tokens), shared by the kernels and the C-ABI layer.
#pragma once
#include <cuda_runtime.h>
#include <cstddef>
#include <cstdint>

namespace fp8idx {

constexpr int kLatent = 512;                 // latent values a token (the attention's values)
constexpr int kRope = 64;                    // rotated key values a token
constexpr int kLatentDim = kLatent + kRope;  // key width
constexpr int kAttnKeys = 64;                // keys per tile (one page)
constexpr int kAttnCols = 64;                // (row, head) columns of a unit
constexpr int kAttnMaxHeads = 128;
constexpr int kAttnMaxParts = 256;            // ranges of the tile axis
constexpr int kSpreadGroups = 8;              // groups that are joined by latent_spread_kernel
constexpr int kStatusBadSlot = 16;           // device status bit: a selected slot past the pool

struct LatentStoreParams {
  const uint16_t* c;      // [T, 512] bf16, row stride c_ld
  const uint16_t* k_pe;   // [T, 64] bf16, row stride pe_ld
  int64_t c_ld, pe_ld;
  const int64_t* positions;  // [T]
  const float* cos_sin;      // [max_pos, 64]: 32 cosines, then 32 sines
  int64_t max_pos;
  const int64_t* slot;    // [T]
  int64_t num_slots;
  int64_t T;
  uint16_t* kv;           // bf16 pool [num_slots, 576], or NULL
  uint8_t* codes;         // fp8 pool [num_slots, 512]
  float* scales;          // [num_slots]
  uint16_t* pe;           // [num_slots, 64]
  const uint16_t* q_pe;   // [T, H, 64] bf16 with strides, or NULL
  uint16_t* q_out;
  int64_t q_row, q_head, o_row, o_head;
  int H;
};

cudaError_t launch_latent_store(const LatentStoreParams& p, bool interleaved, cudaStream_t st);

struct LatentAttnParams {
  const uint16_t* q;        // [rows, H, 576] bf16, strides q_row and q_head
  int64_t q_row, q_head;
  const uint8_t* kv;        // bf16 pool [num_slots, 576] or fp8 codes [num_slots, 512]
  const float* s;           // fp8: [num_slots]
  const uint8_t* pe;        // fp8: [num_slots, 64] bf16
  int64_t num_slots;
  const int32_t* slots;     // selected form: [rows, topk], row stride ld_slots
  int64_t ld_slots;
  int topk;
  const int32_t* block_table;  // paged form: [groups, max_blocks]
  const int32_t* seq_lens;     // [groups]
  int max_blocks;
  int groups;               // query rows (selected form) or requests (paged form)
  int R, H;                 // rows of a group, heads of a row
  float scale_log2;         // softmax scale * log2(e)
  uint16_t* out;            // [rows, H, 512] bf16
  float* lse;               // [rows, H] or NULL
  // schedule: the groups' tiles back to back, cut into `parts` equal ranges;
  // CTA x takes column block x % ncg of range x / ncg
  int ncg, parts;
  int min_tiles;            // tiles a range holds at least, where there are that many
  int whole_groups;         // selected form: ranges end with groups, none is cut
  int* status;
  float* part_o;            // [grid][2][64 x 512] unnormalised sums of cut groups
  float2* part_ml;          // [grid][2][64] (reference maximum in log2 units, sum)
  int4* meta;               // [grid] (group, pieces) of the cut group whose first piece the CTA holds, status bits
  int2* group_meta;         // [groups x ncg] (first CTA, pieces), where groups <= kSpreadGroups
  unsigned long long wait_limit_ns;
  int debug_withhold_first_tile;
};

cudaError_t launch_latent_attn(const LatentAttnParams& p, bool fp8, bool paged, cudaStream_t st);

}  // namespace fp8idx
