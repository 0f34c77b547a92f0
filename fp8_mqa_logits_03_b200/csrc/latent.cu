// latent.cu -- latent attention (absorbed form) for sm_100a: queries against
// one shared 576-value key a token, whose first 512 values are also its value.
//
//   x[c,j]  = scale * q[c,:] . k[j,:]            over the keys j the column sees
//   out[c]  = sum_j exp(x[c,j] - m_c) k[j,0:512] / l_c,   l_c = sum_j exp(x[c,j] - m_c)
//   lse[c]  = m_c + log l_c                      (0 and -inf for a column that sees no key)
//
// for every column c = (query row, head).  The keys of a row are the pool
// slots in a list (selected form) or all tokens of a request through its
// block table (paged form, R rows a request, row t of a request of length L
// sees keys [0, L - R + t + 1)).
//
// Work is cut into units of 64 columns of one group (a query row, or a
// request's R x H columns) times tiles of 64 keys (a page).  The groups' tiles
// lie back to back on one axis, which is cut into ranges, one per CTA: equal
// ones, so that every SM gets the same number of tiles whatever the groups'
// lengths, or, where that costs little, ranges that end with groups (selected
// form) or shares of a group's own (few, short ones).  A group that lies
// inside one range is written directly; one that is cut leaves partial sums
// in 32 bits, which latent_combine_kernel or latent_spread_kernel joins in
// key order: the same bits every time.
//
// One CTA per SM, warp-specialised (448 threads, 227 KB of shared memory):
//   eight warps  softmax: warpgroup w has keys [32 w, 32 w + 32) of a tile,
//                each warp 16 columns of them, four lanes a column.  Scores
//                come from TMEM, running maximum and sum stay in registers,
//                weights go to shared memory; at a segment's end they read
//                the sums from TMEM, divide and write.
//   four warps   producers: gather the tile's key rows into one of two stages
//                in the 128-byte swizzle.  bf16: 16-byte asynchronous copies.
//                fp8: the codes land in one half of the stage and become fp16
//                in its whole, exactly; the rotated part stays bf16.
//   two warps    one issues the score products, part by part as a tile lands,
//                the other the value products.
// Scores: M = 64 columns, N = 64 keys, K = 576.  Values, transposed so that
// the sums of all 512 values fit in half of TMEM: M = 128 values (the same
// key rows read as an MN-major operand), N = 64 columns, K = 64 keys.  The
// weights take the place of the rotated part, which only the scores read.
//
// What bounds it: shared memory's 128 bytes a cycle.  A tile's score products
// read 36 x 4 KB (measured: 33 cycles each, which M = 64 on half of the tensor
// core would take too), its value products 16 x 6 KB (49 cycles; the tensor
// core alone would need 32), its keys are written once, 72 KB: 2500 cycles.
// 4096 rows x 64 heads x 2048 bf16 keys take 1.46 ms (800 TFLOP/s) in a graph of
// three calls and 1.60 ms (730) back to back, where the power limit lowers the
// clock: 2980 cycles a tile with the segments' starts and ends.  fp8 codes are
// written, read and written again (another 64 KB) and take about 3800 (1024
// rows x 128 heads: 0.94 ms either way).  Stages of 64 keys are the largest of
// which two fit beside the queries; over one tile or two, waits for memory and
// hand-overs count: one row of 16 heads x 2048 keys, a tile a CTA, takes 10.6 us
// in a graph, 10.9 a call.  Long contexts with 64 columns a request reach 5.5
// TB/s of keys in a graph of three calls (0.91 ms), 4.6 back to back (1.09).
#include <cstdint>

#include "kernels.cuh"
#include "latent.cuh"
#include "ptx.cuh"
#include "wait.cuh"

namespace fp8idx {

namespace {

constexpr int kStages = 2;
constexpr int kChunks = 9;                      // 64-value (128-byte) chunks of a key row
constexpr int kChunkBytes = kAttnKeys * 128;    // [64 keys][64 values] bf16, swizzled
constexpr int kStageBytes = kChunks * kChunkBytes;
constexpr int kParts = 5;                       // barriers of a stage: four chunk pairs, and the rotated part
constexpr int kInfo = 4;                        // tile descriptions in flight
// The kernel's shape for a kind of pool.
template <bool FP8>
struct Shape {
  static constexpr int kSwg = 2;                  // softmax warpgroups, each with 64 / kSwg of a tile's keys
  static constexpr int kSoftmax = 128 * kSwg;
  static constexpr int kProducers = 128;
  static constexpr int kThreads = kSoftmax + kProducers + 64;
  static constexpr int kFull = FP8 ? 5 : 2;       // announcements of a tile's parts
  // the parts that announcement f covers (fp8: 2, 3, 0, 1, 4, as they are converted)
  __host__ __device__ static constexpr int first_part(int f) { return FP8 ? (f < 4 ? (f + 2) & 3 : f) : (f == 0 ? 0 : f == 1 ? 2 : 5); }
  __host__ __device__ static constexpr int end_part(int f) { return FP8 ? first_part(f) + 1 : (f == 0 ? 2 : 5); }
};
constexpr int kMaxThreads = 448;
static_assert(Shape<true>::kThreads <= kMaxThreads && Shape<false>::kThreads <= kMaxThreads, "threads");

// shared memory, from a 1024-byte boundary
constexpr int kOffQ = 0;
constexpr int kOffK = kStageBytes;              // the 64 query columns take as much as a stage
constexpr int kOffX = kOffK + kStages * kStageBytes;  // softmax warps: maxima and sums exchanged, output transposed
constexpr int kOffMisc = kOffX + kChunkBytes;
constexpr int kMiscBytes = 3 * 1024;
constexpr int kSmemBytes = kOffMisc + kMiscBytes;
static_assert(kSmemBytes <= 227 * 1024, "shared memory per CTA");

// TMEM columns
constexpr uint32_t kTmemO = 0;                  // four blocks of 128 values x 64 columns
constexpr uint32_t kTmemS = 256;                // two score buffers of 64 columns
constexpr uint32_t kTmemPe = 384;               // fp8: the rotated part's scores, two buffers

// What a CTA pays for a second segment (queries, first maxima, sums written
// and joined), in tiles; and the even share above which it does not matter.
// (7 requests x 3 rows of up to 5000 fp8 keys: 39 us in even ranges, 31 in own ones.)
constexpr int kSegmentTiles = 4, kGroupedTiles = 32;

// A running maximum that grows by less than this many powers of two leaves
// the sums as they are: weights may then reach 2^8, which bf16 and the fp32
// sums hold with the same relative precision, and rescaling is rare.
constexpr float kRescaleLog2 = 8.0f;

enum : int { kFirst = 1, kLast = 2, kNull = 4, kEnd = 8, kDirect = 16 };

struct Info {
  unsigned long long mask;  // keys of the tile that exist
  int flags;
  int group;
  int ends;   // paged: keys of the tile that row 0 sees (row t sees t more); large otherwise
  int piece;  // partial-sum slot of a cut group
};

struct Misc {
  uint64_t full[kStages][kParts];
  uint64_t empty[kStages][kParts];
  uint64_t q_full;
  uint64_t s_full[2], s_empty[2];
  uint64_t p_full[2], pv_done[2];  // by tile parity: a wait for a tile never meets the phase of another
  uint64_t drain;
  Info info[kInfo];
  float scale[2][3][kAttnKeys];  // fp8: the tile's key scales s, log2 s and 1 / s, by tile parity
  float q_scale[2][kAttnCols];   // fp8: what a column's scores are multiplied by (log2 units)
  float stat_m[kAttnCols], stat_l[kAttnCols];
  uint32_t unfit[8];  // paged: by softmax warp, keys among 32 whose values it found not finite
  uint32_t tmem;
  int abort_flag;
  int status;       // device status bits of this CTA
  int2 cut;         // (group, pieces) of the cut group whose first piece this CTA holds
  int scan[kMaxThreads / 32];
  int start_group, start_tile, end_tile, pieces;  // paged: where this CTA's range begins (and ends, with pieces > 0)
  int tries[8];
};
static_assert(sizeof(Misc) <= kMiscBytes, "misc");

// ---------------------------------------------------------------- PTX

__device__ __forceinline__ void mma_16(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                         uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// bf16 x bf16 (or f16 x f16) -> f32; a_mn: A is MN-major (B is K-major).
__host__ __device__ constexpr uint32_t idesc_16_f32(int M, int N, bool a_mn, bool f16) {
  return (1u << 4) | ((f16 ? 0u : 1u) << 7) | ((f16 ? 0u : 1u) << 10) | ((a_mn ? 1u : 0u) << 15) | (static_cast<uint32_t>(N >> 3) << 17) |
         (static_cast<uint32_t>(M >> 4) << 24);
}

// MN-major operand in the 128-byte swizzle: rows of 64 values (128 bytes) per
// k, eight k a 1024-byte group, groups back to back; the next 64 values of M
// lie one chunk further.
__device__ __forceinline__ uint64_t smem_desc_mn_sw128(uint32_t saddr) {
  uint64_t d = 0;
  d |= static_cast<uint64_t>((saddr >> 4) & 0x3FFF);
  d |= static_cast<uint64_t>(kChunkBytes >> 4) << 16;  // between 64-value blocks of M
  d |= static_cast<uint64_t>(1024 >> 4) << 32;         // between groups of eight k
  d |= static_cast<uint64_t>(1) << 46;
  d |= static_cast<uint64_t>(2) << 61;
  return d;
}

// 16 lanes x 16 (or 32) columns: thread t receives, for each 8-column block j, columns
// 8j + 2(t % 4) + {0, 1} of lane t / 4 in r[4j], r[4j+1] and of lane t / 4 + 8
// in r[4j+2], r[4j+3].
__device__ __forceinline__ void tmem_ld_16(uint32_t taddr, uint32_t (&r)[8]) {
  asm volatile("tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(taddr)
               : "memory");
}

__device__ __forceinline__ void tmem_ld_16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}

// 32 lanes x 16 consecutive columns, one lane a thread.
__device__ __forceinline__ void tmem_ld_x16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_st_x16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15};" ::"r"(r[0]),
      "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
      "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// 16-byte asynchronous copy; `bytes` 0 writes zeros and reads nothing.
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(reinterpret_cast<uint64_t>(src)),
               "r"(bytes)
               : "memory");
}
// One arrival on `bar` once this thread's earlier asynchronous copies have landed.
__device__ __forceinline__ void cp_async_arrive(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}
// The same for 4 bytes.
__device__ __forceinline__ void cp_async4(uint32_t dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(reinterpret_cast<uint64_t>(src)),
               "r"(bytes)
               : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void cp_async_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }
// Orders this thread's view of generic-proxy writes before later async-proxy
// (tensor core) reads of the same shared memory.
__device__ __forceinline__ void fence_async_shared() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

__device__ __forceinline__ uint4 ld_shared16(uint32_t src) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(src)
               : "memory");
  return v;
}
__device__ __forceinline__ void st_shared16(uint32_t dst, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(dst), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}

// The e4m3 codes in the lower and upper half of w as fp16 pairs (exact).
__device__ __forceinline__ void e4m3x4_f16(uint32_t w, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(w));
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
// The larger of each pair of 16-bit halves.
__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.u16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
// Four 8 x 8 matrices of 16-bit values, each stored transposed: this lane
// gives the address of one 16-byte row.
__device__ __forceinline__ void stmatrix_x4_trans(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b),
               "r"(c), "r"(d)
               : "memory");
}

// The same, stored as they are.
__device__ __forceinline__ void stmatrix_x4(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c),
               "r"(d)
               : "memory");
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint64_t pack_u32x2(uint32_t lo, uint32_t hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "r"(lo), "r"(hi));
  return r;
}
__device__ __forceinline__ void unpack_u32x2(uint64_t v, uint32_t& lo, uint32_t& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=r"(lo), "=r"(hi) : "l"(v));
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// A bounded wait by a whole warp; true only where every lane's wait
// succeeded.  (Polling without suspending was slower: the warps that wait
// took the shared-memory pipe from those that work.)
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, volatile int* abort_flag, int* status,
                                          unsigned long long limit_ns) {
  return __all_sync(0xFFFFFFFFu, wait_phase<kSpin>(bar, parity, abort_flag, status, limit_ns));
}

// One lane of a converged warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(p));
  return p != 0;
}

// ---------------------------------------------------------------- schedule

// Tiles of group g: at least one, so that an empty group is written too.
template <bool PAGED>
__device__ __forceinline__ int group_len(const LatentAttnParams& p, int g) {
  if (!PAGED) return p.topk;
  const int L = __ldg(p.seq_lens + g);
  return max(0, min(L, p.max_blocks * kPageSize));  // (max_blocks * 64 is checked to fit)
}
__device__ __forceinline__ int tiles_of(int len) { return max(1, (len + kAttnKeys - 1) / kAttnKeys); }

// Keys of a tile that not every row of the group sees (those from `ends` on),
// and whose values are not finite: 0 * value would not be 0 in the rows that
// must not see them, so their values become 0 (and an fp8 pool's 1 / scale, for
// the weights' sums).  The values themselves tell: a score that is not finite
// may be the query's doing, and its other rows see the key as it is.  All eight
// softmax warps call this, a thread looks at a quarter of a key.  Returns the
// first such key (128: none).  Out of line: it is rare.
template <bool FP8>
__device__ __noinline__ int drop_unfit_keys(Misc& ms, uint8_t* stage, int b, uint32_t parity, int ends, volatile int* abort_flag,
                                             unsigned long long limit) {
#pragma unroll 1
  for (int u = 0; u < Shape<FP8>::kFull; ++u)  // the tile landed long ago; this is for the thread's own view of it
    warp_wait(&ms.full[b][u], parity, abort_flag, &ms.status, limit);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, key = (warp & 1) * 32 + lane;
  uint8_t* krow = stage + (warp >> 1) * 2 * kChunkBytes + key * 128;
  constexpr uint32_t kInf = FP8 ? 0x7C00u : 0x7F80u;  // exponent bits of fp16, bf16
  bool unfit = FP8 && !(fabsf(ms.scale[b][0][key]) < INFINITY);
#pragma unroll 1
  for (int x = 0; x < 16; ++x) {
    const uint4 v = *reinterpret_cast<const uint4*>(krow + (x >> 3) * kChunkBytes + (x & 7) * 16);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const uint32_t y = (&v.x)[e];
      unfit = unfit || (y & kInf) == kInf || ((y >> 16) & kInf) == kInf;
    }
  }
  const uint32_t found = __ballot_sync(0xFFFFFFFFu, unfit && key >= ends);
  if (lane == 0) ms.unfit[warp] = found;
  named_bar_sync(2, Shape<FP8>::kSoftmax);
  const uint32_t all = ms.unfit[warp & 1] | ms.unfit[2 + (warp & 1)] | ms.unfit[4 + (warp & 1)] | ms.unfit[6 + (warp & 1)];
  if ((all >> lane) & 1) {
#pragma unroll 1
    for (int x = 0; x < 16; ++x)
      *reinterpret_cast<uint4*>(krow + (x >> 3) * kChunkBytes + (x & 7) * 16) = make_uint4(0, 0, 0, 0);
    if (FP8 && warp < 2) ms.scale[b][2][key] = 0.f;
  }
  const uint32_t lo = ms.unfit[0] | ms.unfit[2] | ms.unfit[4] | ms.unfit[6];
  const uint32_t hi = ms.unfit[1] | ms.unfit[3] | ms.unfit[5] | ms.unfit[7];
  return lo ? __ffs(lo) - 1 : hi ? 31 + __ffs(hi) : kAttnKeys + kPageSize;
}

}  // namespace

// ---------------------------------------------------------------- the kernel

template <bool PAGED, bool FP8>
__global__ void __launch_bounds__(Shape<FP8>::kThreads, 1) latent_attn_kernel(const __grid_constant__ LatentAttnParams p) {
  using Sh = Shape<FP8>;
  constexpr int kThreads = Sh::kThreads, kSoftmax = Sh::kSoftmax, kSwg = Sh::kSwg, kProducers = Sh::kProducers;
  constexpr int kScoreWarp = kThreads / 32 - 2, kValueWarp = kThreads / 32 - 1;
  extern __shared__ __align__(1024) uint8_t smem[];
  Misc& ms = *reinterpret_cast<Misc*>(smem + kOffMisc);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int cg = blockIdx.x % p.ncg, part = blockIdx.x / p.ncg;
  volatile int* abort_flag = &ms.abort_flag;
  const unsigned long long limit = p.wait_limit_ns;

  if (tid == 0) {
    for (int s = 0; s < kStages; ++s)
      for (int i = 0; i < kParts; ++i) {
        // codes: one arrival a warp; asynchronous copies: one a thread (bf16: and one with the tile's description)
        mbar_init(&ms.full[s][i], FP8 && i < 4 ? kProducers / 32 : kProducers + (!FP8 && i == 0 ? 1 : 0));
        mbar_init(&ms.empty[s][i], 1);
      }
    mbar_init(&ms.q_full, kProducers);
    for (int b = 0; b < 2; ++b) {
      mbar_init(&ms.s_full[b], 1);
      mbar_init(&ms.s_empty[b], kSoftmax);
      mbar_init(&ms.p_full[b], kSoftmax);
      mbar_init(&ms.pv_done[b], 1);
    }
    mbar_init(&ms.drain, 2);
    ms.abort_flag = 0;
    ms.status = 0;
    ms.cut = make_int2(0, 0);
    fence_mbar_init();
  }
  if (warp == kScoreWarp) {
    tmem_alloc(&ms.tmem, 512);
    tmem_relinquish();
  }

  griddep_wait();  // the inputs are ready, and nobody reads this workspace any more

  // ---- this CTA's range of the tile axis
  bool too_long = false;
  int64_t total;
  // Paged: few requests with little work each get CTAs of their own, as many as
  // a request takes at `tau` tiles each, so that no CTA has the end of one and
  // the start of another (each segment costs about as much as kSegmentTiles
  // tiles).  tau is the smallest of eight values from the even share on whose
  // CTAs suffice; where it is more than the even share and a segment, the even
  // ranges are the shorter ones.
  const int even_of = p.parts, tries = 8;
  auto tau_at = [&](int even, int u) {
    const int tau0 = max(even, p.min_tiles);
    return tau0 + u * max(1, tau0 / 8);
  };
  if (PAGED && p.groups <= 32) {
    // a request a lane, in every warp alike: no barrier
    const int L = lane < p.groups ? __ldg(p.seq_lens + lane) : 0;
    too_long = L > p.max_blocks * kPageSize;
    const int mine = lane < p.groups ? tiles_of(max(0, min(L, p.max_blocks * kPageSize))) : 0;
    const int all = __reduce_add_sync(0xFFFFFFFFu, mine), even = (all + even_of - 1) / even_of;
    total = all;
    int tau = 0;
    if (p.groups <= p.parts && even <= kGroupedTiles) {
#pragma unroll 1
      for (int u = 0; u < tries && tau == 0; ++u) {
        const int v = tau_at(even, u);
        if (v > max(even + kSegmentTiles, p.min_tiles)) break;
        if (static_cast<int>(__reduce_add_sync(0xFFFFFFFFu, (mine + v - 1) / v)) <= p.parts) tau = v;
      }
    }
    // the requests' shares of the CTAs, or of the tile axis
    const int c = tau > 0 ? (mine + tau - 1) / tau : mine;
    int pre = c;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int v = __shfl_up_sync(0xFFFFFFFFu, pre, d);
      if (lane >= d) pre += v;
    }
    const int64_t parts = min(static_cast<int64_t>(p.parts), total);
    const int x = tau > 0 ? part : part < parts ? static_cast<int>(part * total / parts) : all;
    if (warp == 0) {
      if (lane == 0) ms.pieces = tau > 0 ? 0 : -1;
      __syncwarp();
      if (x >= pre - c && x < pre) {
        const int r = x - (pre - c);
        ms.start_group = lane;
        ms.start_tile = tau > 0 ? static_cast<int>(static_cast<int64_t>(r) * mine / c) : r;
        if (tau > 0) {
          ms.end_tile = static_cast<int>(static_cast<int64_t>(r + 1) * mine / c);
          ms.pieces = c;
        }
      }
    }
  } else if (PAGED) {
    // prefix sum over the requests: each thread a contiguous run of them
    const int per = (p.groups + kThreads - 1) / kThreads;
    const int g0 = min(tid * per, p.groups), g1 = min(g0 + per, p.groups);
    int mine = 0;
    for (int g = g0; g < g1; ++g) {
      mine += tiles_of(group_len<true>(p, g));
      too_long = too_long || __ldg(p.seq_lens + g) > p.max_blocks * kPageSize;
    }
    auto scan = [&](int v) {  // inclusive, over the block
      int inc = v;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int o = __shfl_up_sync(0xFFFFFFFFu, inc, d);
        if (lane >= d) inc += o;
      }
      if (lane == 31) ms.scan[warp] = inc;
      __syncthreads();
      for (int w = 0; w < warp; ++w) inc += ms.scan[w];
      return inc;
    };
    const int inc = scan(mine);
    int all = 0;
    for (int w = 0; w < kThreads / 32; ++w) all += ms.scan[w];
    total = all;
    const int even = (all + even_of - 1) / even_of;
    int tau = 0;
    if (p.groups <= min(p.parts, kThreads) && even <= kGroupedTiles) {
      if (tid < tries) ms.tries[tid] = 0;
      __syncthreads();
#pragma unroll
      for (int u = 0; u < tries; ++u) {
        const int v = tau_at(even, u), c = __reduce_add_sync(0xFFFFFFFFu, (mine + v - 1) / v);
        if (lane == 0) atomicAdd(&ms.tries[u], c);
      }
      __syncthreads();
      for (int u = tries - 1; u >= 0; --u)
        if (ms.tries[u] <= p.parts) tau = tau_at(even, u);
      if (tau > max(even + kSegmentTiles, p.min_tiles)) tau = 0;
    }
    if (tau > 0) {
      const int c = (mine + tau - 1) / tau;
      if (tid == 0) ms.pieces = 0;
      const int r = part - (scan(c) - c);
      if (r >= 0 && r < c) {
        ms.start_group = tid;
        ms.start_tile = static_cast<int>(static_cast<int64_t>(r) * mine / c);
        ms.end_tile = static_cast<int>(static_cast<int64_t>(r + 1) * mine / c);
        ms.pieces = c;
      }
    } else {
      if (tid == 0) ms.pieces = -1;
      const int64_t parts = min(static_cast<int64_t>(p.parts), total);
      const int64_t x = part < parts ? part * total / parts : total;
      int at = inc - mine;  // the run's first tile
      if (x >= at && x < at + mine) {
        for (int g = g0; g < g1; ++g) {
          const int n = tiles_of(group_len<true>(p, g));
          if (x < at + n) {
            ms.start_group = g;
            ms.start_tile = static_cast<int>(x - at);
            break;
          }
          at += n;
        }
      }
    }
  } else {
    total = static_cast<int64_t>(p.groups) * tiles_of(p.topk);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const int64_t parts = min(static_cast<int64_t>(p.parts), total);
  int64_t x0 = part < parts ? part * total / parts : 0;
  int64_t x1 = part < parts ? (part + 1) * total / parts : 0;
  if (PAGED && ms.pieces >= 0) {  // a request's own CTAs
    x0 = 0;
    x1 = ms.pieces > 0 ? ms.end_tile - ms.start_tile : 0;
  }
  if (!PAGED && p.whole_groups) {  // ranges that end with groups
    x0 = static_cast<int64_t>(part) * p.groups / p.parts * tiles_of(p.topk);
    x1 = static_cast<int64_t>(part + 1) * p.groups / p.parts * tiles_of(p.topk);
  }
  const uint32_t tbase = ms.tmem;
  if (too_long) atomicOr(&ms.status, kStatusSeqLenTooLong);

  if (warp >= kSoftmax / 32 && warp < kScoreWarp) {
    // ================================================================ producers
    constexpr int kRows = kProducers / 8, NK = kAttnKeys / kRows;  // rows side by side, rows a thread
    const int pt = tid - kSoftmax;
    const int piece = pt & 7, r0 = pt >> 3;  // 16-byte piece of a chunk row; rows r0 + kRows k
    const uint32_t row_dst = smem_u32(smem + kOffK) + r0 * 128;
    const uint32_t swz = (piece ^ (r0 & 7)) << 4;
    // fp8: 16 codes become pieces 2 (piece % 4) and the next of chunk piece / 4;
    // lanes of the second chunk write the odd piece first, so that the eight
    // lanes of a row hit eight different 16-byte bank groups
    const int odd = piece >> 2, sub = 2 * (piece & 3);
    const uint32_t fdst0 = odd * kChunkBytes + (((sub + odd) ^ (r0 & 7)) << 4);
    const uint32_t fdst1 = odd * kChunkBytes + (((sub + 1 - odd) ^ (r0 & 7)) << 4);
    constexpr int kRowBytes = FP8 ? kLatent : kLatentDim * 2;

    // ---- where the stream stands: the next tile to look at is tile t of group g
    int g, t, te = 0, len = 0;
    bool direct = false, from_start = false, fresh = true;  // fresh: no tile of the segment has been emitted
    int left = static_cast<int>(x1 - x0);  // tiles of this CTA's range behind the current segment
    const int32_t* list = nullptr;
    int bad = 0;
    int next_idx[2] = {-1, -1};         // raw list entries of its keys lane and lane + 32 (paged: the page)
    if (PAGED) {
      g = ms.start_group;
      t = ms.start_tile;
    } else {
      const int per = tiles_of(p.topk);
      g = static_cast<int>(x0 / per);
      t = static_cast<int>(x0 - static_cast<int64_t>(g) * per);
    }
    // Starts the segment of group g at tile t.
    auto open_segment = [&]() {
      len = group_len<PAGED>(p, g);
      const int nt = tiles_of(len);
      te = min(nt, t + left);
      direct = t == 0 && te == nt;
      fresh = true;
      if (t == 0 && te < nt && pt == 0) {
        // the group goes on in the ranges after this one, up to the one that holds its last tile
        int pieces = PAGED ? ms.pieces : 0;
        if (pieces <= 0) {
          const int64_t last = x1 - left + nt - 1;
          pieces = static_cast<int>(((last + 1) * parts - 1) / total) - part + 1;
        }
        ms.cut = make_int2(g, pieces);
      }
      from_start = t == 0;
      if (t == 0 && pt == 0 && p.groups <= kSpreadGroups)
        p.group_meta[g * p.ncg + cg] = make_int2(static_cast<int>(blockIdx.x), te < nt ? ms.cut.y : 1);
      list = PAGED ? p.block_table + static_cast<int64_t>(g) * p.max_blocks
                   : p.slots + static_cast<int64_t>(g) * p.ld_slots;
      left -= te - t;
    };
    auto fetch_idx = [&]() {
      if (PAGED) {
        next_idx[0] = t < te && t * kAttnKeys < len ? __ldg(list + t) : -1;  // a tile is a page
      } else {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int j = t * kAttnKeys + h * 32 + lane;
          next_idx[h] = t < te && j < len ? __ldg(list + j) : -1;
        }
      }
    };

    // ---- the tile about to be written
    Info d;
    int key_slot = -1;       // fp8: pool slot of key pt
    int row[NK];             // pool slots of its rows r0 + kRows k, -1 where there is none
    const int num_slots = static_cast<int>(p.num_slots), num_pages = num_slots / kPageSize;
    // Finds the next tile that holds keys (or ends a segment, or the stream) and describes it in d.
    auto advance = [&]() {
      for (;;) {
        if (t == te) {
          if (left == 0) {
            d.flags = kEnd;
            return;
          }
          ++g;
          t = 0;
          open_segment();
          fetch_idx();
        }
        int sl[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          int v = -1;
          if (PAGED) {
            const int pg = next_idx[0];
            if (t * kAttnKeys + h * 32 + lane < len) {
              if (pg >= 0 && pg < num_pages) v = pg * kPageSize + h * 32 + lane;
              else bad |= kStatusBadPage;
            }
          } else {
            v = next_idx[h];
            if (v >= num_slots) {
              v = -1;
              bad |= kStatusBadSlot;
            }
          }
          sl[h] = v;
        }
        d.mask = __ballot_sync(0xFFFFFFFFu, sl[0] >= 0) |
                 (static_cast<unsigned long long>(__ballot_sync(0xFFFFFFFFu, sl[1] >= 0)) << 32);
        const bool last = t == te - 1, null = d.mask == 0;
        d.flags = (fresh ? kFirst : 0) | (last ? kLast : 0) | (null ? kNull : 0) | (direct ? kDirect : 0);
        d.group = g;
        d.ends = PAGED ? len - p.R + 1 - t * kAttnKeys : 1 << 20;
        d.piece = static_cast<int>(blockIdx.x) * 2 + (from_start ? 1 : 0);
        ++t;
        fetch_idx();
        if (null && !last) continue;  // nothing to do and nothing to say
        if (!null) {
          fresh = false;
#pragma unroll
          for (int k = 0; k < NK; ++k) {
            row[k] = __shfl_sync(0xFFFFFFFFu, sl[kRows * k >> 5], (r0 + kRows * k) & 31);
          }
          if (FP8 && pt < kAttnKeys) key_slot = pt < 32 ? sl[0] : sl[1];
        }
        return;
      }
    };
    auto row_at = [&](int v) { return p.kv + static_cast<int64_t>(max(v, 0)) * kRowBytes + piece * 16; };
    // fp8: 16 codes of part c, row r0 + kRows k, into the stage as fp16.
    auto store_codes = [&](const uint4& v, int c, int k, uint32_t dst) {
      const uint32_t rd = dst + k * (kRows * 128) + 2 * c * kChunkBytes;
      uint32_t a[4], b[4];
      e4m3x4_f16(v.x, a[0], a[1]);
      e4m3x4_f16(v.y, a[2], a[3]);
      e4m3x4_f16(v.z, b[0], b[1]);
      e4m3x4_f16(v.w, b[2], b[3]);
      st_shared16(rd + fdst0, odd ? b[0] : a[0], odd ? b[1] : a[1], odd ? b[2] : a[2], odd ? b[3] : a[3]);
      st_shared16(rd + fdst1, odd ? a[0] : b[0], odd ? a[1] : b[1], odd ? a[2] : b[2], odd ? a[3] : b[3]);
    };

    // ---- the group's query columns
    auto copy_q = [&](int group) {
      const int cols = p.R * p.H;
#pragma unroll
      for (int k = 0; k < NK; ++k) {
        const int col = cg * kAttnCols + r0 + kRows * k;
        const bool v = col < cols;
        const int qr = PAGED && v ? col / p.H : 0, h = v ? col - qr * p.H : 0;
        const uint8_t* qs = reinterpret_cast<const uint8_t*>(
            p.q + (static_cast<int64_t>(group) * p.R + qr) * p.q_row + h * p.q_head) + piece * 16;
        const uint32_t qd = smem_u32(smem + kOffQ) + (r0 + kRows * k) * 128 + swz;
#pragma unroll
        for (int c = 0; c < kChunks; ++c) cp_async16(qd + c * kChunkBytes, qs + c * 128, v ? 16 : 0);
      }
    };
    // fp8: the codes are products' other side in fp16, so a column becomes
    // fp16 too, in place, times the power of two that brings its largest value
    // next to 2^14: exact but for values 2^28 times smaller, whose error
    // (2^-39 of the largest) is below the fp32 sum's.  The rotated part meets
    // bf16 and stays bf16.  A thread converts the pieces that it copied.
    auto convert_q = [&](float (&fac)[NK]) {
      cp_async_wait_all();
#pragma unroll
      for (int k = 0; k < NK; ++k) fac[k] = 0.f;
#pragma unroll 1
      for (int k = 0; k < NK; ++k) {
        if (cg * kAttnCols + kRows * k >= p.R * p.H) break;  // no such columns (zeros)
        const uint32_t at = smem_u32(smem + kOffQ) + (r0 + kRows * k) * 128 + swz;
        uint4 v[kChunks];
        uint32_t top = 0;  // largest magnitudes of the two halves of a word
#pragma unroll
        for (int c = 0; c < kChunks; ++c) {
          v[c] = ld_shared16(at + c * kChunkBytes);
#pragma unroll
          for (int e = 0; e < 4; ++e) top = max_u16x2(top, (&v[c].x)[e] & 0x7FFF7FFFu);
        }
        top = max(top & 0xFFFFu, top >> 16);
        top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
        top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
        top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 4));
        const int ex = top >> 7;  // biased exponent of the largest value
        // times 2^(140 - ex), at most 2^126 so that its inverse is an ordinary
        // number too; a zero or non-finite column stays
        const int up = ex == 0 || ex == 255 ? 0 : min(140 - ex, 126);
        const float f = __uint_as_float(static_cast<uint32_t>(127 + up) << 23);
        const float back = p.scale_log2 * __uint_as_float(static_cast<uint32_t>(127 - up) << 23);
#pragma unroll
        for (int u = 0; u < NK; ++u)
          if (u == k) fac[u] = back;
#pragma unroll
        for (int c = 0; c < kChunks; ++c) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const uint32_t y = (&v[c].x)[e];
            const float lo = __uint_as_float(y << 16) * f, hi = __uint_as_float(y & 0xFFFF0000u) * f;
            (&v[c].x)[e] = c < 8 ? pack_f16(lo, hi) : pack_bf16(lo, hi);
          }
          st_shared16(at + c * kChunkBytes, v[c].x, v[c].y, v[c].z, v[c].w);
        }
      }
      mbar_arrive(&ms.q_full);
    };

    bool ok = true;
    if (left > 0) {
      open_segment();
      fetch_idx();
      // on its way while the first list entries are; used if tile 0 holds keys (it is then of this group)
      copy_q(g);
    } else {
      t = te;
    }
    advance();
    for (int i = 0; ok; ++i) {
      const int st = i & 1;
      const uint32_t ph = (i >> 1) & 1;
      const int flags = d.flags;
      const bool null = flags & (kNull | kEnd);
      // The group's query columns; their place is free once the scores of tile
      // i - 1 are done (and of tile i - 2: a tile i - 1 without keys has none).
      const bool first = (flags & kFirst) && !null;
      auto next_q = [&]() {
        if (!warp_wait(&ms.s_full[st ^ 1], ((i - 1) >> 1) & 1, abort_flag, &ms.status, limit)) return false;
        if (i > 1 && !warp_wait(&ms.s_full[st], ph ^ 1, abort_flag, &ms.status, limit)) return false;
        copy_q(d.group);
        return true;
      };
      if (i == 0 && null) cp_async_wait_all();  // the queries copied ahead are not used: out of the way of the next ones
      if (!FP8 && first) {
        if (i > 0 && !next_q()) break;
        cp_async_arrive(&ms.q_full);
      }
      // ---- describe the tile.  The entry was tile i - 4's; the values of
      // tile i - 2 have begun, so every role is past tile i - 4.
      if (!warp_wait(&ms.empty[st][0], ph ^ 1, abort_flag, &ms.status, limit)) break;
      if (pt == 0) {
        ms.info[i & (kInfo - 1)] = d;
        if (!FP8) mbar_arrive(&ms.full[st][0]);
      }
      const bool withhold = p.debug_withhold_first_tile && i == 0;
      const uint32_t dst = row_dst + st * kStageBytes;
      if (FP8 && !null) {
        // The codes land in the first half of the stage, and the rotated part,
        // bf16 as it is, in its place: parts 2 and 3 in part 0's, 0 and 1 in
        // part 1's.  They become fp16 in this order, each as it lands, in its own
        // place, which for the last two is where the ones before have landed.  A
        // row's eight pieces are one warp's, landing and converted.
        const uint32_t land = dst + swz;
        if (pt < kAttnKeys) cp_async4(smem_u32(&ms.scale[st][0][pt]), p.s + max(key_slot, 0), key_slot >= 0 ? 4 : 0);
#pragma unroll
        for (int u = 0; u < 4; ++u) {  // part (u + 2) % 4 into chunk u
          if (u == 2 && !warp_wait(&ms.empty[st][1], ph ^ 1, abort_flag, &ms.status, limit)) { ok = false; break; }
#pragma unroll
          for (int k = 0; k < NK; ++k)
            cp_async16(land + u * kChunkBytes + k * (kRows * 128), row_at(row[k]) + ((u + 2) & 3) * 128, row[k] >= 0 ? 16 : 0);
          cp_async_commit();
        }
        if (!ok) break;
        if (!warp_wait(&ms.empty[st][2], ph ^ 1, abort_flag, &ms.status, limit) ||
            !warp_wait(&ms.empty[st][3], ph ^ 1, abort_flag, &ms.status, limit) ||
            !warp_wait(&ms.empty[st][4], ph ^ 1, abort_flag, &ms.status, limit))
          break;
#pragma unroll
        for (int k = 0; k < NK; ++k)
          cp_async16(land + 8 * kChunkBytes + k * (kRows * 128),
                     p.pe + static_cast<int64_t>(max(row[k], 0)) * (kRope * 2) + piece * 16, row[k] >= 0 ? 16 : 0);
        cp_async_arrive(&ms.full[st][4]);
        cp_async_commit();
        if (first) {  // the queries, while the codes are on their way
          if (i > 0 && !next_q()) break;
          float qfac[NK];
          convert_q(qfac);
          if (piece == 0) {
#pragma unroll
            for (int k = 0; k < NK; ++k) ms.q_scale[st][r0 + kRows * k] = qfac[k];
          }
        }
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          if (u == 0) cp_async_wait<4>();
          else if (u == 1) cp_async_wait<3>();
          else if (u == 2) cp_async_wait<2>();
          else cp_async_wait<1>();
          if (u == 0 && pt < kAttnKeys) {
            // a scale of 0 (or below 2^-60, or of a key that does not exist)
            // counts as 2^-60: its log and inverse are used
            const float x = ms.scale[st][0][pt], y = x < 8.673617379884035e-19f ? 8.673617379884035e-19f : x;
            ms.scale[st][0][pt] = y;
            ms.scale[st][1][pt] = log2f(y);
            ms.scale[st][2][pt] = 1.f / y;
          }
          uint4 raw[NK];
#pragma unroll
          for (int k = 0; k < NK; ++k) raw[k] = ld_shared16(land + u * kChunkBytes + k * (kRows * 128));
          if (u == 3) __syncwarp();  // (this part's own place)
#pragma unroll
          for (int k = 0; k < NK; ++k) store_codes(raw[k], (u + 2) & 3, k, dst);
          __syncwarp();
          if (lane == 0 && !(withhold && u == 0)) mbar_arrive(&ms.full[st][u]);
        }
      } else if (FP8) {
        // nothing to bring: every thread arrives for the rotated part, a warp for the others
        for (int f = 0; f < Sh::kFull; ++f) {
          if (f > 0 && (flags & kEnd)) break;
          if (!(flags & kEnd) && !warp_wait(&ms.empty[st][Sh::first_part(f)], ph ^ 1, abort_flag, &ms.status, limit)) { ok = false; break; }
          __syncwarp();
          if (f == 4 || lane == 0) mbar_arrive(&ms.full[st][f]);
        }
      } else {
#pragma unroll
        for (int f = 0; f < Sh::kFull; ++f) {
          if (f > 0 && (flags & kEnd)) break;
#pragma unroll
          for (int c = Sh::first_part(f); c < Sh::end_part(f); ++c) {
            if (c > 0 && !(flags & kEnd) &&
                !warp_wait(&ms.empty[st][c], ph ^ 1, abort_flag, &ms.status, limit)) { ok = false; break; }
            if (null) continue;
#pragma unroll
            for (int u = 0; u < (c < 4 ? 2 : 1); ++u)
#pragma unroll
              for (int k = 0; k < NK; ++k)
                cp_async16(dst + (2 * c + u) * kChunkBytes + k * (kRows * 128) + swz, row_at(row[k]) + (2 * c + u) * 128,
                           row[k] >= 0 ? 16 : 0);
          }
          if (!ok) break;
          if (null) mbar_arrive(&ms.full[st][f]);
          else if (!(withhold && f == 0)) cp_async_arrive(&ms.full[st][f]);
        }
      }
      if (!ok) break;
      if (flags & kEnd) break;
      advance();
    }
    cp_async_wait_all();
    if (bad) atomicOr(&ms.status, bad);
  } else if (warp == kScoreWarp) {
    // ================================================================ score products
    // A whole warp runs the issue loops, so that descriptors and branches are
    // uniform, and one elected lane issues: MMAs issued from a branch on the
    // lane number took 280 cycles each, elected ones 32 (scores) and 49.
    constexpr uint32_t id_s = idesc_16_f32(64, 64, false, FP8), id_pe = idesc_16_f32(64, 64, false, false);
    const uint64_t q_d = smem_desc_k128_sw128(smem_u32(smem + kOffQ));
    int nq = 0;  // query loads seen
    for (int i = 0;; ++i) {
      const int st = i & 1;
      const uint32_t ph = (i >> 1) & 1;
      const uint64_t k_d = smem_desc_k128_sw128(smem_u32(smem + kOffK + st * kStageBytes));
      if (!warp_wait(&ms.s_empty[st], ph ^ 1, abort_flag, &ms.status, limit)) break;
      if (!warp_wait(&ms.full[st][0], ph, abort_flag, &ms.status, limit)) break;
      const int flags = ms.info[i & (kInfo - 1)].flags;
      if (flags & (kNull | kEnd)) {
        bool ok = true;
        for (int c = 1; c < Sh::kFull && ok && !(flags & kEnd); ++c)
          ok = warp_wait(&ms.full[st][c], ph, abort_flag, &ms.status, limit);
        if (!ok) break;
        if (elect_one()) {
          mbar_arrive(&ms.s_full[st]);
        }
        __syncwarp();
        if (flags & kEnd) break;
        continue;
      }
      if (flags & kFirst) {
        if (!warp_wait(&ms.q_full, nq & 1, abort_flag, &ms.status, limit)) break;
        ++nq;
        fence_async_shared();  // other threads wrote the queries
      }
      bool ok = true;
#pragma unroll
      for (int f = 0; f < Sh::kFull; ++f) {
        if (f > 0 && !warp_wait(&ms.full[st][f], ph, abort_flag, &ms.status, limit)) { ok = false; break; }
        // the rows were written by other threads
        fence_async_shared();
        tc_fence_after();
        if (elect_one()) {
#pragma unroll
          for (int c = Sh::first_part(f); c < Sh::end_part(f); ++c) {
            const uint32_t dd = tbase + (FP8 && c == 4 ? kTmemPe : kTmemS) + st * 64;
#pragma unroll
            for (int ks = 0; ks < (c < 4 ? 8 : 4); ++ks) {
              const int off = ((2 * c + (ks >> 2)) * kChunkBytes + (ks & 3) * 32) >> 4;
              mma_16(dd, q_d + off, k_d + off, c == 4 ? id_pe : id_s,
                     ks > 0 || (c != Sh::first_part(0) && !(FP8 && c == 4)));
            }
          }
          if (f == Sh::kFull - 1) mma_commit(&ms.s_full[st]);
        }
        __syncwarp();
      }
      if (!ok) break;
    }
    if (elect_one()) mma_commit(&ms.drain);
    __syncwarp();
  } else if (warp == kValueWarp) {
    // ================================================================ value products
    // (as many columns as there are, in sixteens: the sums of the others are never read)
    const uint32_t id_v = idesc_16_f32(128, (min(kAttnCols, p.R * p.H - cg * kAttnCols) + 15) & ~15, true, FP8);
    for (int i = 0;; ++i) {
      const int st = i & 1;
      if (!warp_wait(&ms.p_full[st], (i >> 1) & 1, abort_flag, &ms.status, limit)) break;
      const int flags = ms.info[i & (kInfo - 1)].flags;
      if (flags & kEnd) break;
      tc_fence_after();
      if (elect_one()) {
        if (flags & kNull) {
#pragma unroll
          for (int c = 0; c < kParts - 1; ++c) mbar_arrive(&ms.empty[st][c]);
          mbar_arrive(&ms.pv_done[st]);
          mbar_arrive(&ms.empty[st][4]);
        } else {
          const uint64_t v_d = smem_desc_mn_sw128(smem_u32(smem + kOffK + st * kStageBytes));
          const uint64_t p_d = smem_desc_k128_sw128(smem_u32(smem + kOffK + st * kStageBytes + 8 * kChunkBytes));
#pragma unroll
          for (int c = 0; c < 4; ++c) {
#pragma unroll
            for (int ks = 0; ks < 4; ++ks)
              mma_16(tbase + kTmemO + c * 64, v_d + ((2 * c * kChunkBytes + ks * 2048) >> 4), p_d + ks * 2, id_v,
                       ks > 0 || !(flags & kFirst));
            if (c < 3) mma_commit(&ms.empty[st][c]);
          }
          mma_commit(&ms.pv_done[st]);  // no later than the stage's last release
          mma_commit(&ms.empty[st][3]);
          mma_commit(&ms.empty[st][4]);  // (the weights lie in the rotated part's place)
        }
      }
      __syncwarp();
    }
    if (elect_one()) mma_commit(&ms.drain);
    __syncwarp();
  } else if (warp < kSoftmax / 32) {
    // ================================================================ softmax and output
    const int wg = warp >> 2, quad = warp & 3;                     // keys [kKeys wg, + kKeys); TMEM lane quadrant
    constexpr int kKeys = 64 / kSwg, NJ = kKeys / 8, NR = 4 * NJ;  // keys, 8-key blocks, scores a thread
    const uint32_t lane_base = static_cast<uint32_t>(quad) << 21;  // TMEM lane 32 * quad
    const int rr = quad * 16 + (lane >> 2);        // this thread's columns (heads): rr and rr + 8
    const int cq = kKeys * wg + 2 * (lane & 3);    // its keys: 8 j + cq + {0, 1}
    const int cols = p.R * p.H;
    int trow[2];                             // row within the group of each column
#pragma unroll
    for (int h = 0; h < 2; ++h) trow[h] = PAGED ? min((cg * kAttnCols + rr + 8 * h) / p.H, p.R - 1) : 0;
    // fp8: weights are fp16, whose range the maximum is moved away from the
    // lower end of (2^7 next to it, 2^15 before a rescale; 2^-24 is the smallest)
    constexpr float kBias = FP8 ? 7.f : 0.f;
    // exchanged between the two warpgroups
    float* half_max = reinterpret_cast<float*>(smem + kOffX);
    float* stat_l1 = half_max;
    const uint32_t prow = smem_u32(smem + kOffK + 8 * kChunkBytes) + (quad * 16 + (lane & 15)) * 128;  // weights: this lane's row to store
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
    float to_log2[2] = {p.scale_log2, p.scale_log2};
    bool dead = false;
    for (int i = 0;; ++i) {
      const int b = i & 1;
      // a wait that gave up is carried to the votes below, so that all
      // warps leave together
      if (!warp_wait(&ms.s_full[b], (i >> 1) & 1, abort_flag, &ms.status, limit)) dead = true;
      tc_fence_after();
      const Info& f = ms.info[i & (kInfo - 1)];
      const int flags = dead ? kNull : f.flags;
      const bool end = flags & kEnd;
      if (flags & kFirst) {
        m[0] = m[1] = -INFINITY;
        l[0] = l[1] = 0.f;
        if (FP8) {
          to_log2[0] = ms.q_scale[b][rr];
          to_log2[1] = ms.q_scale[b][rr + 8];
        }
      }
      uint32_t w[2 * NJ], r[NR];
      float mx[2] = {-INFINITY, -INFINITY}, la[2];
      bool suspect = false;  // paged: the score of a key that its row must not see is not finite
      // The tile's scores (fp8: in log2 units, with the keys' scales), unseen ones -inf, and this thread's maxima.
      auto read_scores = [&]() {
        tmem_ld_16(tbase + kTmemS + b * 64 + wg * kKeys + lane_base, r);
        if (FP8) {
          // (codes . q) s + rotated part, in log2 units, plus log2 s: the
          // weight of key j is exp2 of this, i.e. it carries the key's scale
          const uint64_t tl2[2] = {pack_f32x2(to_log2[0], to_log2[0]), pack_f32x2(to_log2[1], to_log2[1])};
#pragma unroll
          for (int half = 0; half < NJ / 4; ++half) {  // 32 columns at a time
            uint32_t e[16];
            tmem_ld_16(tbase + kTmemPe + b * 64 + wg * kKeys + half * 32 + lane_base, e);
            tmem_ld_wait();
#pragma unroll
            for (int jj = 0; jj < 4; ++jj) {
              const int j = half * 4 + jj;
              const uint64_t v2 = *reinterpret_cast<const uint64_t*>(&ms.scale[b][0][8 * j + cq]);
              const uint64_t g2 = *reinterpret_cast<const uint64_t*>(&ms.scale[b][1][8 * j + cq]);
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                const int x = 4 * j + 2 * h, y = 4 * jj + 2 * h;
                uint64_t z = fma_f32x2(pack_u32x2(r[x], r[x + 1]), v2, pack_u32x2(e[y], e[y + 1]));
                z = fma_f32x2(z, tl2[h], g2);
                unpack_u32x2(z, r[x], r[x + 1]);
              }
            }
          }
        } else {
          tmem_ld_wait();
        }
        const unsigned long long mask = f.mask;
        const int ends = f.ends;
        mx[0] = mx[1] = -INFINITY;
        const bool whole = mask == ~0ull && ends >= kAttnKeys;
        if (!whole) {
          // bit 8 j + e: key 8 j + cq + e exists, and row h sees it
          const unsigned long long here = mask >> cq;
          unsigned long long sees[2];
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int lim = ends + trow[h];  // keys of the tile that the row sees
            sees[h] = (lim >= kAttnKeys ? mask : lim <= 0 ? 0ull : mask & ((1ull << lim) - 1)) >> cq;
          }
#pragma unroll
          for (int j = 0; j < NR; ++j) {
            const int h = (j >> 1) & 1, bit = 8 * (j >> 2) + (j & 1);
            const bool real = (here >> bit) & 1, seen = (sees[h] >> bit) & 1;
            // the key, or the query: drop_unfit_keys tells
            if (PAGED && real && !seen && !(fabsf(__uint_as_float(r[j])) < INFINITY)) suspect = true;
            if (!seen) r[j] = 0xFF800000u;
          }
        }
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
          mx[0] = fmaxf(mx[0], fmaxf(__uint_as_float(r[4 * j]), __uint_as_float(r[4 * j + 1])));
          mx[1] = fmaxf(mx[1], fmaxf(__uint_as_float(r[4 * j + 2]), __uint_as_float(r[4 * j + 3])));
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) mx[h] = (FP8 ? mx[h] : mx[h] * to_log2[h]) - kBias;
      };
      // The weights of this thread's keys, with the reference maxima as they
      // are, and their sums (packed pairs of keys).
      auto weigh = [&]() {
        uint64_t neg2[2], la2[2] = {0, 0}, tl2[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float neg = m[h] == -INFINITY ? 0.f : -m[h];
          neg2[h] = pack_f32x2(neg, neg);
          tl2[h] = pack_f32x2(to_log2[h], to_log2[h]);
        }
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
          uint64_t inv2;
          if (FP8) inv2 = *reinterpret_cast<const uint64_t*>(&ms.scale[b][2][8 * j + cq]);
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint64_t x2 = pack_u32x2(r[4 * j + 2 * h], r[4 * j + 2 * h + 1]);
            float a, c;
            unpack_f32x2(FP8 ? add_f32x2(x2, neg2[h]) : fma_f32x2(x2, tl2[h], neg2[h]), a, c);
            a = ex2(a);
            c = ex2(c);
            la2[h] = FP8 ? fma_f32x2(pack_f32x2(a, c), inv2, la2[h]) : add_f32x2(pack_f32x2(a, c), la2[h]);
            w[2 * j + h] = FP8 ? pack_f16(a, c) : pack_bf16(a, c);
          }
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          float a, c;
          unpack_f32x2(la2[h], a, c);
          la[h] = a + c;
        }
      };
      auto put_weights = [&]() {  // two 8-key blocks of the warp's 16 columns at a time
#pragma unroll
        for (int j = 0; j < NJ; j += 2)
          stmatrix_x4(prow + b * kStageBytes + (((wg * NJ + j + (lane >> 4)) ^ (lane & 7)) << 4), w[2 * j], w[2 * j + 1],
                      w[2 * j + 2], w[2 * j + 3]);
      };
      const bool live = !(flags & (kNull | kEnd));
      // Pass 0: the weights with the maxima as they are (not on a segment's
      // first tile, which has none), and one vote: whether some score outgrew
      // its column's reference maximum, the end, a wait that gave up.  Mostly
      // none did, and the weights stand.  Else pass 1: new maxima, the sums so
      // far scaled to them, and the weights again.
      // (Pass 1 reads the scores once more: kept over the vote, they would spill.)
      bool leave = false;
#pragma unroll 1
      for (int pass = 0; pass < 2; ++pass) {
        if (live && (pass == 1 || !(flags & kFirst))) read_scores();
        if (pass == 1) {
          // (the sums hold still once the previous value product is done)
          if (i > 0 && !warp_wait(&ms.pv_done[b ^ 1], ((i - 1) >> 1) & 1, abort_flag, &ms.status, limit)) dead = true;
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            mx[h] = fmaxf(mx[h], __shfl_xor_sync(0xFFFFFFFFu, mx[h], 1));
            mx[h] = fmaxf(mx[h], __shfl_xor_sync(0xFFFFFFFFu, mx[h], 2));
          }
          if ((lane & 3) == 0) {
            half_max[wg * kAttnCols + rr] = mx[0];
            half_max[wg * kAttnCols + rr + 8] = mx[1];
          }
          if (!PAGED || p.R == 1) {  // (one row a request: it sees every key that exists)
            named_bar_sync(2, kSoftmax);
          } else if (bar_red_or(2, kSoftmax, suspect)) {
            const int first = drop_unfit_keys<FP8>(ms, smem + kOffK + b * kStageBytes, b, (i >> 1) & 1, f.ends, abort_flag, limit);
            // a row that sees such a key gives NaN, also where its score is -inf (a weight of 0, times a value that is gone)
#pragma unroll
            for (int h = 0; h < 2; ++h)
              if (first < f.ends + trow[h]) l[h] = __uint_as_float(0x7FC00000u);
          }
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            mx[h] = fmaxf(mx[h], half_max[(wg ^ 1) * kAttnCols + rr + 8 * h]);
            float fac = 1.f;
            if (flags & kFirst) {
              m[h] = mx[h];
            } else if (mx[h] > m[h] + kRescaleLog2) {
              fac = ex2(m[h] - mx[h]);
              m[h] = mx[h];
              l[h] *= fac;
            }
            if ((lane & 3) == 0 && wg == 0) ms.stat_m[rr + 8 * h] = fac;
          }
          if (!(flags & kFirst)) {
            named_bar_sync(2, kSoftmax);
            tc_fence_after();
#pragma unroll 1
            for (int c = wg; c < 16; c += kSwg) {
              uint32_t o[16];
              tmem_ld_x16(tbase + kTmemO + c * 16 + lane_base, o);
              tmem_ld_wait();
#pragma unroll
              for (int k = 0; k < 16; ++k)
                o[k] = __float_as_uint(__uint_as_float(o[k]) * ms.stat_m[(c & 3) * 16 + k]);
              tmem_st_x16(tbase + kTmemO + c * 16 + lane_base, o);
            }
            tmem_st_wait();
          }
          named_bar_sync(2, kSoftmax);  // the factors are read before they are written again
        }
        const bool weighs = live && (pass == 1 || !(flags & kFirst));
        if (weighs) weigh();
        if (weighs) put_weights();
        if (pass == 1) break;
        const bool grow = mx[0] > m[0] + kRescaleLog2 || mx[1] > m[1] + kRescaleLog2 || (PAGED && suspect);
        const bool vote = bar_red_or(1, kSoftmax, dead || end || grow);
        if (vote && bar_red_or(1, kSoftmax, dead || end)) {
          leave = true;
          break;
        }
        if (!live || !(vote || (flags & kFirst))) break;
      }
      if (leave) {
        mbar_arrive(&ms.p_full[b]);  // the value warp sees the end too
        break;
      }
      if (!dead) {
        tc_fence_before();
        mbar_arrive(&ms.s_empty[b]);
      }
      if (live) {
        l[0] += la[0];
        l[1] += la[1];
        fence_async_shared();
      }
      tc_fence_before();
      mbar_arrive(&ms.p_full[b]);
      if (!(flags & kLast)) continue;

      // ---- the segment's end: its sums, divided (a whole group) or as they are (a cut one)
      const int group = f.group, slot = f.piece;
      const bool none = (flags & kNull) && (flags & kFirst);  // no key at all: the sums were never written
      const bool direct = flags & kDirect;
      // (a last tile without keys is done at once, the one before it perhaps not)
      if (i > 0 && !warp_wait(&ms.pv_done[b ^ 1], ((i - 1) >> 1) & 1, abort_flag, &ms.status, limit)) dead = true;
      if (!warp_wait(&ms.pv_done[b], (i >> 1) & 1, abort_flag, &ms.status, limit)) dead = true;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        l[h] += __shfl_xor_sync(0xFFFFFFFFu, l[h], 1);
        l[h] += __shfl_xor_sync(0xFFFFFFFFu, l[h], 2);
        if ((lane & 3) == 0) {
          if (wg == 0) ms.stat_m[rr + 8 * h] = m[h];
          (wg == 0 ? ms.stat_l : stat_l1)[rr + 8 * h] = l[h];
        }
      }
      if (bar_red_or(1, kSoftmax, dead)) break;
      tc_fence_after();
      const int n = min(kAttnCols, cols - cg * kAttnCols);
      const int64_t col0 = static_cast<int64_t>(group) * cols + cg * kAttnCols;
      if (tid < kAttnCols) {
        const float mm = ms.stat_m[tid], ll = ms.stat_l[tid] + stat_l1[tid];
        if (tid < n) {
          if (!direct) p.part_ml[static_cast<int64_t>(slot) * kAttnCols + tid] = make_float2(mm, ll);
          else if (p.lse) p.lse[col0 + tid] = (mm + log2f(ll)) * 0.69314718055994531f;
        }
        if (direct) ms.stat_l[tid] = ll == 0.f ? 0.f : 1.f / ll;
      }
      named_bar_sync(2, kSoftmax);
      if (direct) {
        // This warpgroup's 32 columns: 32 values x 16 columns at a time,
        // divided, rounded, transposed through the warp's part of the exchange
        // buffer, and written as 64 bytes a column by four lanes.
        const int cb = wg * 32;
        uint8_t* tb = smem + kOffX + warp * 1024;  // [16 columns][32 values], pieces swizzled
        const int mcol = (lane & 7) + (lane >> 4) * 8, mhalf = (lane >> 3) & 1;  // stmatrix: this lane's column, value half
        uint16_t* oo = p.out + (col0 + cb) * kLatent + quad * 32;
        if (cb < n) {
          uint32_t o[16], ahead[16];
          // block c: values 128 (c / 2) + 32 quad + {0 .. 31}, columns cb + 16 (c % 2) + {0 .. 15}
          auto fetch = [&](int c) {
            uint32_t (&lo)[8] = *reinterpret_cast<uint32_t(*)[8]>(&ahead[0]);
            uint32_t (&hi)[8] = *reinterpret_cast<uint32_t(*)[8]>(&ahead[8]);
            const uint32_t at = tbase + kTmemO + (c >> 1) * 64 + cb + (c & 1) * 16 + lane_base;
            tmem_ld_16(at, lo);
            tmem_ld_16(at + (16u << 16), hi);
          };
          if (none) {
#pragma unroll
            for (int k = 0; k < 16; ++k) ahead[k] = 0;
          } else {
            fetch(0);
          }
#pragma unroll 1
          for (int c = 0; c < 8; ++c) {
            if (cb + (c & 1) * 16 >= n) continue;
            tmem_ld_wait();
#pragma unroll
            for (int k = 0; k < 16; ++k) o[k] = ahead[k];
            if (!none) {
              const int next = c + 1 < 8 && cb + ((c + 1) & 1) * 16 >= n ? c + 2 : c + 1;
              if (next < 8) fetch(next);
            }
            const float2 i0 = *reinterpret_cast<const float2*>(&ms.stat_l[cb + (c & 1) * 16 + 2 * (lane & 3)]);
            const float2 i1 = *reinterpret_cast<const float2*>(&ms.stat_l[cb + (c & 1) * 16 + 8 + 2 * (lane & 3)]);
            uint32_t w4[8];  // [value half][16-lane half's 8 rows][column block]
#pragma unroll
            for (int v = 0; v < 2; ++v) {
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                const int e = 8 * v + 2 * h;
                w4[4 * v + h] = pack_bf16(__uint_as_float(o[e]) * i0.x, __uint_as_float(o[e + 1]) * i0.y);
                w4[4 * v + 2 + h] = pack_bf16(__uint_as_float(o[e + 4]) * i1.x, __uint_as_float(o[e + 5]) * i1.y);
              }
            }
            __syncwarp();
#pragma unroll
            for (int v = 0; v < 2; ++v)
              stmatrix_x4_trans(smem_u32(tb) + mcol * 64 + (((2 * v + mhalf) ^ ((mcol >> 1) & 3)) << 4), w4[4 * v],
                                w4[4 * v + 1], w4[4 * v + 2], w4[4 * v + 3]);
            __syncwarp();
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              const int col = k * 8 + (lane >> 2), part = lane & 3;
              const uint4 v = *reinterpret_cast<const uint4*>(tb + col * 64 + ((part ^ ((col >> 1) & 3)) << 4));
              const int cc = (c & 1) * 16 + col;
              if (cb + cc < n)
                *reinterpret_cast<uint4*>(oo + static_cast<int64_t>(cc) * kLatent + (c >> 1) * 128 + part * 8) = v;
            }
          }
        }
      } else {
        // [slot][value block, column half][column quad][value][column of the quad]
        float* po = p.part_o + (static_cast<int64_t>(slot) * 64 * 128 + quad * 32 + lane) * 4;
        // block t: values 128 (t / 2) + 32 quad + lane, columns 32 wg + 16 (t % 2) + {0 .. 15}
        if (wg * 32 < n) {
          uint32_t o[16], ahead[16];
          if (none) {
#pragma unroll
            for (int k = 0; k < 16; ++k) ahead[k] = 0;
          } else {
            tmem_ld_x16(tbase + kTmemO + wg * 32 + lane_base, ahead);
          }
#pragma unroll 1
          for (int t = 0; t < 8; ++t) {
            tmem_ld_wait();
#pragma unroll
            for (int k = 0; k < 16; ++k) o[k] = ahead[k];
            if (!none && t < 7)
              tmem_ld_x16(tbase + kTmemO + ((t + 1) >> 1) * 64 + wg * 32 + ((t + 1) & 1) * 16 + lane_base, ahead);
#pragma unroll
            for (int j = 0; j < 4; ++j)
              if (wg * 32 + (t & 1) * 16 + 4 * j < n)
                *reinterpret_cast<uint4*>(po + (((t >> 1) * 2 + wg) * 8 + (t & 1) * 4 + j) * 512) =
                    make_uint4(o[4 * j], o[4 * j + 1], o[4 * j + 2], o[4 * j + 3]);
          }
        }
      }
      tc_fence_before();
      named_bar_sync(2, kSoftmax);  // stat_m and stat_l are read before the next group writes them
    }
  }
  if (warp == kScoreWarp) {
    // every MMA issued has finished before shared memory and TMEM go away
    const uint64_t td = global_timer_ns();
    while (!mbar_try_wait(&ms.drain, 0) && global_timer_ns() - td < 200000000ull) {
    }
  }
  tc_fence_before();
  __syncthreads();
  if (tid == 0) p.meta[blockIdx.x] = make_int4(ms.cut.x, ms.cut.y, ms.status, 0);
  if (warp == kScoreWarp) {
    tc_fence_after();
    tmem_dealloc(tbase, 512);
  }
}

// ---------------------------------------------------------------- joining cut groups
//
// A cut group's pieces lie in the CTAs x, x + ncg, ..., in key order: the first
// in its second slot, the others in their first.  With (m_k, l_k, O_k) the
// pieces' reference maxima, sums and unnormalised results,
//   w_k = 2^(m_k - max m) / sum_k l_k 2^(m_k - max m),   out = sum_k w_k O_k.
// Bound by latency: the pieces come from L2 (at most two a CTA, 128 KB each
// with 64 columns).

__device__ __forceinline__ int64_t piece_slot(int x, int k, int ncg) {
  return static_cast<int64_t>(x + k * ncg) * 2 + (k == 0 ? 1 : 0);
}

// The call's status block: every CTA's bits.
__device__ __forceinline__ void collect_status(const LatentAttnParams& p) {
  int bits = 0;
  for (int k = threadIdx.x; k < p.parts * p.ncg; k += blockDim.x) bits |= p.meta[k].z;
  bits = (__syncthreads_or(bits & kStatusWaitTimeout) ? kStatusWaitTimeout : 0) |
         (__syncthreads_or(bits & kStatusBadPage) ? kStatusBadPage : 0) |
         (__syncthreads_or(bits & kStatusSeqLenTooLong) ? kStatusSeqLenTooLong : 0) |
         (__syncthreads_or(bits & kStatusBadSlot) ? kStatusBadSlot : 0);
  if (threadIdx.x < kStatusBytes / 4) p.status[threadIdx.x] = threadIdx.x == 0 ? bits : 0;
}

__device__ __forceinline__ float4 piece_at(const LatentAttnParams& p, int64_t slot, int vb, int quad, int val) {
  return *reinterpret_cast<const float4*>(p.part_o + slot * (kAttnCols * kLatent) +
                                          ((vb * 2 + (quad >> 3)) * 8 + (quad & 7)) * 512 + val * 4);
}
__device__ __forceinline__ void fma4(float4& acc, const float4& v, const float4& w) {
  acc.x = fmaf(v.x, w.x, acc.x);
  acc.y = fmaf(v.y, w.y, acc.y);
  acc.z = fmaf(v.z, w.z, acc.z);
  acc.w = fmaf(v.w, w.w, acc.w);
}
__device__ __forceinline__ void write4(const LatentAttnParams& p, const float4& acc, int64_t oc, int n, int quad, int vb,
                                       int val) {
#pragma unroll
  for (int e = 0; e < 4; ++e)
    if (4 * quad + e < n)
      p.out[(oc + 4 * quad + e) * kLatent + vb * 128 + val] = static_cast<uint16_t>(pack_bf16((&acc.x)[e], 0.f));
}

// The usual form: a group has been cut in two or three, and there are up to a
// group per CTA.  Block (x, y): the group whose first piece CTA x holds, value
// block y, all columns: two sets of 128 threads (one value each) take every
// second column quad, all their loads of a piece under way at once.
constexpr int kJoinThreads = 256, kJoinChunk = 32;

__global__ void __launch_bounds__(kJoinThreads) latent_combine_kernel(const __grid_constant__ LatentAttnParams p) {
  __shared__ float4 wt[kJoinChunk][kAttnCols / 4];
  __shared__ float2 top_inv[kAttnCols];
  griddep_wait();
  const int tid = threadIdx.x;
  if (blockIdx.x == 0 && blockIdx.y == 0) collect_status(p);
  const int4 mt = p.meta[blockIdx.x];
  const int np = mt.y, x = blockIdx.x, vb = blockIdx.y;
  if (np < 2) return;
  const int cols = p.R * p.H, cg = x % p.ncg;
  const int n = min(kAttnCols, cols - cg * kAttnCols), quads = (n + 3) / 4;
  const int64_t oc = static_cast<int64_t>(mt.x) * cols + cg * kAttnCols;
  const int sub = tid >> 7, val = tid & 127;
  float4 acc[8], ahead[8];
#pragma unroll
  for (int u = 0; u < 8; ++u) {
    acc[u] = make_float4(0.f, 0.f, 0.f, 0.f);
    if (sub + 2 * u < quads) ahead[u] = piece_at(p, piece_slot(x, 0, p.ncg), vb, sub + 2 * u, val);
  }
  {
    // four lanes a column: the largest reference and the sum over all pieces
    const int c = tid >> 2, part = tid & 3;
    float top = -INFINITY, sum = 0.f;
    if (c < n) {
#pragma unroll 4
      for (int k = part; k < np; k += 4) top = fmaxf(top, p.part_ml[piece_slot(x, k, p.ncg) * kAttnCols + c].x);
    }
    top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
    top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
    const float ref = top == -INFINITY ? 0.f : top;
    if (c < n) {
#pragma unroll 4
      for (int k = part; k < np; k += 4) {
        const float2 ml = p.part_ml[piece_slot(x, k, p.ncg) * kAttnCols + c];
        sum = fmaf(ml.y, exp2f(ml.x - ref), sum);
      }
    }
    sum += __shfl_xor_sync(0xFFFFFFFFu, sum, 1);
    sum += __shfl_xor_sync(0xFFFFFFFFu, sum, 2);
    if (part == 0 && c < n) {
      top_inv[c] = make_float2(ref, sum == 0.f ? 0.f : 1.f / sum);
      if (vb == 0 && p.lse) p.lse[oc + c] = (top + log2f(sum)) * 0.69314718055994531f;
    }
  }
  for (int k0 = 0; k0 < np; k0 += kJoinChunk) {
    const int nk = min(kJoinChunk, np - k0);
    __syncthreads();
    for (int e = tid; e < nk * kAttnCols; e += kJoinThreads) {
      const int k = e / kAttnCols, c = e % kAttnCols;
      if (c < n) {
        const float2 ti = top_inv[c];
        (&wt[k][c >> 2].x)[c & 3] = exp2f(p.part_ml[piece_slot(x, k0 + k, p.ncg) * kAttnCols + c].x - ti.x) * ti.y;
      }
    }
    __syncthreads();
    for (int k = 0; k < nk; ++k) {
      float4 v[8];
#pragma unroll
      for (int u = 0; u < 8; ++u) v[u] = ahead[u];
      if (k0 + k + 1 < np) {
#pragma unroll
        for (int u = 0; u < 8; ++u)
          if (sub + 2 * u < quads) ahead[u] = piece_at(p, piece_slot(x, k0 + k + 1, p.ncg), vb, sub + 2 * u, val);
      }
#pragma unroll
      for (int u = 0; u < 8; ++u)
        if (sub + 2 * u < quads) fma4(acc[u], v[u], wt[k][sub + 2 * u]);
    }
  }
#pragma unroll
  for (int u = 0; u < 8; ++u)
    if (sub + 2 * u < quads) write4(p, acc[u], oc, n, sub + 2 * u, vb, val);
}

// The form for few groups (at most kSpreadGroups, so each may be cut into many
// pieces).  Block (x, y): group x / ncg, column block x % ncg, value block
// y % 4, column quad y / 4.  Four sets of 128 threads take every fourth piece,
// and their sums are joined; the first loads go out before the weights are known.
constexpr int kSpreadThreads = 512, kSpreadAhead = 8;

__global__ void __launch_bounds__(kSpreadThreads) latent_spread_kernel(const __grid_constant__ LatentAttnParams p) {
  __shared__ float4 wt[kAttnMaxParts];
  __shared__ float4 acc_of[3][128];
  griddep_wait();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (blockIdx.x == 0 && blockIdx.y == 0) collect_status(p);
  const int2 e = p.group_meta[blockIdx.x];
  const int x = e.x, np = e.y;
  // (a CTA that gave up has not written the entries of the groups that it never
  // reached: what is there instead must not be followed out of the workspace)
  if (np < 2 || x < 0 || x + static_cast<int64_t>(np - 1) * p.ncg >= static_cast<int64_t>(p.parts) * p.ncg) return;
  const int cols = p.R * p.H, cg = blockIdx.x % p.ncg;
  const int n = min(kAttnCols, cols - cg * kAttnCols);
  const int quad = blockIdx.y >> 2, vb = blockIdx.y & 3;
  if (4 * quad >= n) return;
  const int64_t oc = static_cast<int64_t>(blockIdx.x / p.ncg) * cols + cg * kAttnCols;
  const int sub = tid >> 7, val = tid & 127;
  float4 first[kSpreadAhead];
#pragma unroll
  for (int u = 0; u < kSpreadAhead; ++u)
    if (sub + 4 * u < np) first[u] = piece_at(p, piece_slot(x, sub + 4 * u, p.ncg), vb, quad, val);
  if (warp < 4) {
    // warp w: the weights of column 4 quad + w in every piece
    const int col = 4 * quad + warp;
    float2 ml[kAttnMaxParts / 32];
    float top = -INFINITY;
#pragma unroll
    for (int u = 0; u < kAttnMaxParts / 32; ++u) {
      const int k = lane + 32 * u;
      ml[u] = col < n && k < np ? p.part_ml[piece_slot(x, k, p.ncg) * kAttnCols + col] : make_float2(-INFINITY, 0.f);
      top = fmaxf(top, ml[u].x);
    }
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, d));
    const float ref = top == -INFINITY ? 0.f : top;
    float sum = 0.f;
#pragma unroll
    for (int u = 0; u < kAttnMaxParts / 32; ++u) {
      ml[u].x = exp2f(ml[u].x - ref);
      sum = fmaf(ml[u].y, ml[u].x, sum);
    }
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, d);
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
#pragma unroll
    for (int u = 0; u < kAttnMaxParts / 32; ++u)
      if (lane + 32 * u < np) (&wt[lane + 32 * u].x)[warp] = ml[u].x * inv;
    if (vb == 0 && lane == 0 && p.lse && col < n) p.lse[oc + col] = (top + log2f(sum)) * 0.69314718055994531f;
  }
  __syncthreads();
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
  for (int u = 0; u < kSpreadAhead; ++u)
    if (sub + 4 * u < np) fma4(acc, first[u], wt[sub + 4 * u]);
#pragma unroll 4
  for (int k = sub + 4 * kSpreadAhead; k < np; k += 4) fma4(acc, piece_at(p, piece_slot(x, k, p.ncg), vb, quad, val), wt[k]);
  if (sub > 0) acc_of[sub - 1][val] = acc;
  __syncthreads();
  if (sub > 0) return;
#pragma unroll
  for (int u = 0; u < 3; ++u) {
    const float4 v = acc_of[u][val];
    acc.x += v.x;
    acc.y += v.y;
    acc.z += v.z;
    acc.w += v.w;
  }
  write4(p, acc, oc, n, quad, vb, val);
}

cudaError_t launch_latent_attn(const LatentAttnParams& p, bool fp8, bool paged, cudaStream_t st) {
  const void* kern =
      paged ? (fp8 ? reinterpret_cast<const void*>(latent_attn_kernel<true, true>)
                   : reinterpret_cast<const void*>(latent_attn_kernel<true, false>))
            : (fp8 ? reinterpret_cast<const void*>(latent_attn_kernel<false, true>)
                   : reinterpret_cast<const void*>(latent_attn_kernel<false, false>));
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes);
  if (e != cudaSuccess) return e;
  // Both launches are programmatic dependents: a launch's latency overlaps the
  // end of the kernel before it, whose results it waits for on the device.
  const int grid = p.parts * p.ncg;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(grid));
  cfg.blockDim = dim3(fp8 ? Shape<true>::kThreads : Shape<false>::kThreads);
  cfg.dynamicSmemBytes = kSmemBytes;
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  LatentAttnParams copy = p;
  void* args[] = {&copy};
  e = cudaLaunchKernelExC(&cfg, kern, args);
  if (e != cudaSuccess) return e;
  cfg.dynamicSmemBytes = 0;
  if (p.groups <= kSpreadGroups) {
    cfg.gridDim = dim3(static_cast<unsigned>(p.groups * p.ncg), static_cast<unsigned>(4 * ((min(kAttnCols, p.R * p.H) + 3) / 4)));
    cfg.blockDim = dim3(kSpreadThreads);
    return cudaLaunchKernelExC(&cfg, reinterpret_cast<const void*>(latent_spread_kernel), args);
  }
  // (no group is cut where the ranges end with groups: the status alone)
  cfg.gridDim = p.whole_groups ? dim3(1) : dim3(static_cast<unsigned>(grid), 4);
  cfg.blockDim = dim3(kJoinThreads);
  return cudaLaunchKernelExC(&cfg, reinterpret_cast<const void*>(latent_combine_kernel), args);
}

}  // namespace fp8idx
