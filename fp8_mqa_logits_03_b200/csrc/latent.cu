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
// request's R x H columns) times tiles of 64 keys.  The groups' tiles lie back
// to back on one axis, which is cut into equal ranges, one per CTA: every SM
// gets the same number of tiles whatever the groups' lengths.  A group that
// lies inside one range is written directly; one that is cut leaves partial
// sums, which combine_kernel joins in order.
//
// One CTA, warp-specialised:
//   warps 0-3  softmax: read the 64 x 64 scores from TMEM (16 heads a warp,
//              four lanes a head), running maximum and sum in registers,
//              weights as bf16 into shared memory; at a group's end they read
//              the sums from TMEM, divide and write.
//   warps 4-7  producers: gather the tile's key rows into one of two stages
//              with 16-byte asynchronous copies in the 128-byte swizzle.
//   warp 8     one thread issues the MMAs, whichever is ready: a group of
//              score products as its part of the tile lands, or the value
//              product of a tile whose weights are ready.
// Scores: M = 64 columns, N = 64 keys, K = 576.  Values, transposed so that
// the sums of all 512 values fit in half of TMEM: M = 128 values (the same
// key rows read as an MN-major operand), N = 64 columns, K = 64 keys.
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
constexpr int kProducers = 128;
constexpr int kSoftmax = 128;
constexpr int kThreads = kSoftmax + kProducers + 32;

// shared memory, from a 1024-byte boundary
constexpr int kOffQ = 0;
constexpr int kOffK = kStageBytes;              // the 64 query columns take as much as a stage
constexpr int kOffP = kOffK + kStages * kStageBytes;
constexpr int kOffMisc = kOffP + kChunkBytes;
constexpr int kSmemBytes = kOffMisc + 2048 + 1024;
static_assert(kSmemBytes <= 227 * 1024, "shared memory per CTA");

// TMEM columns
constexpr uint32_t kTmemO = 0;                  // four blocks of 128 values x 64 columns
constexpr uint32_t kTmemS = 256;                // two score buffers of 64 columns
constexpr uint32_t kTmemPe = 384;               // fp8: the rotated part's scores, two buffers

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
  uint64_t p_full, pv_done, drain;
  Info info[kInfo];
  float stat_m[kAttnCols], stat_l[kAttnCols];
  uint32_t tmem;
  int abort_flag;
  int scan[kThreads / 32 + 1];
  int start_group, start_tile;
};
static_assert(sizeof(Misc) <= 2048, "misc");

// ---------------------------------------------------------------- PTX

__device__ __forceinline__ void mma_bf16(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                         uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// bf16 x bf16 -> f32; a_mn: A is MN-major (B is K-major).
__host__ __device__ constexpr uint32_t idesc_bf16_f32(int M, int N, bool a_mn) {
  return (1u << 4) | (1u << 7) | (1u << 10) | ((a_mn ? 1u : 0u) << 15) | (static_cast<uint32_t>(N >> 3) << 17) |
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

// 16 lanes x 64 columns: thread t receives, for each 8-column block j, columns
// 8j + 2(t % 4) + {0, 1} of lane t / 4 in r[4j], r[4j+1] and of lane t / 4 + 8
// in r[4j+2], r[4j+3].
__device__ __forceinline__ void tmem_ld_16x64(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x8.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]),
        "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]),
        "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr)
      : "memory");
}

__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31};" ::"r"(r[0]),
      "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]),
      "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]),
      "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31]), "r"(taddr)
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
__device__ __forceinline__ void cp_async_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }
// Orders this thread's view of generic-proxy writes before later async-proxy
// (tensor core) reads of the same shared memory.
__device__ __forceinline__ void fence_async_shared() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// wait_phase by a whole warp; true only where every lane's wait succeeded.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, volatile int* abort_flag, int* status,
                                          unsigned long long limit_ns) {
  return __all_sync(0xFFFFFFFFu, wait_phase<kSpin>(bar, parity, abort_flag, status, limit_ns));
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

}  // namespace

// ---------------------------------------------------------------- the kernel

template <bool PAGED>
__global__ void __launch_bounds__(kThreads, 1) latent_attn_kernel(const __grid_constant__ LatentAttnParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  Misc& ms = *reinterpret_cast<Misc*>(smem + kOffMisc);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int cg = blockIdx.x % p.ncg, part = blockIdx.x / p.ncg;
  volatile int* abort_flag = &ms.abort_flag;
  const unsigned long long limit = p.wait_limit_ns;

  if (tid == 0) {
    for (int s = 0; s < kStages; ++s)
      for (int i = 0; i < kParts; ++i) {
        mbar_init(&ms.full[s][i], kProducers + (i == 0 ? 1 : 0));  // part 0 also announces the tile's description
        mbar_init(&ms.empty[s][i], 1);
      }
    mbar_init(&ms.q_full, kProducers);
    for (int b = 0; b < 2; ++b) {
      mbar_init(&ms.s_full[b], 1);
      mbar_init(&ms.s_empty[b], kSoftmax);
    }
    mbar_init(&ms.p_full, kSoftmax);
    mbar_init(&ms.pv_done, 1);
    mbar_init(&ms.drain, 1);
    ms.abort_flag = 0;
    fence_mbar_init();
    p.meta[blockIdx.x] = make_int4(0, 0, 0, 0);
  }
  if (warp == 8) {
    tmem_alloc(&ms.tmem, 512);
    tmem_relinquish();
  }

  // ---- this CTA's range of the tile axis
  int64_t total;
  if (PAGED) {
    // prefix sum over the requests: each thread a contiguous run of them
    const int per = (p.groups + kThreads - 1) / kThreads;
    const int g0 = min(tid * per, p.groups), g1 = min(g0 + per, p.groups);
    int mine = 0;
    for (int g = g0; g < g1; ++g) {
      mine += tiles_of(group_len<true>(p, g));
      if (cg == 0 && part == 0 && __ldg(p.seq_lens + g) > static_cast<int64_t>(p.max_blocks) * kPageSize)
        atomicOr(p.status, kStatusSeqLenTooLong);
    }
    int inc = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int v = __shfl_up_sync(0xFFFFFFFFu, inc, d);
      if (lane >= d) inc += v;
    }
    if (lane == 31) ms.scan[warp] = inc;
    __syncthreads();
    int before = 0, all = 0;
    for (int w = 0; w < kThreads / 32; ++w) {
      if (w < warp) before += ms.scan[w];
      all += ms.scan[w];
    }
    total = all;
    const int64_t parts = min(static_cast<int64_t>(p.parts), total);
    const int64_t x = part < parts ? part * total / parts : total;
    int at = before + inc - mine;  // the run's first tile
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
  } else {
    total = static_cast<int64_t>(p.groups) * tiles_of(p.topk);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const int64_t parts = min(static_cast<int64_t>(p.parts), total);
  const int64_t x0 = part < parts ? part * total / parts : 0;
  const int64_t x1 = part < parts ? (part + 1) * total / parts : 0;
  const uint32_t tbase = ms.tmem;

  if (warp >= 4 && warp < 8) {
    // ================================================================ producers
    const int pt = tid - kSoftmax;
    const int piece = pt & 7, r0 = pt >> 3;  // 16-byte piece of a chunk row; rows r0 + 16 k
    const uint32_t dst0 = smem_u32(smem + kOffK) + r0 * 128 + ((piece ^ (r0 & 7)) << 4);
    const uint32_t qdst0 = smem_u32(smem + kOffQ) + r0 * 128 + ((piece ^ (r0 & 7)) << 4);
    int g, t;
    if (PAGED) {
      g = ms.start_group;
      t = ms.start_tile;
    } else {
      const int per = tiles_of(p.topk);
      g = static_cast<int>(x0 / per);
      t = static_cast<int>(x0 - static_cast<int64_t>(g) * per);
    }
    int i = 0;           // tiles emitted
    bool ok = true;
    int bad = 0;
    for (int64_t x = x0; x < x1 && ok; ++g, t = 0) {
      // ---- a segment: tiles [t, te) of group g
      const int len = group_len<PAGED>(p, g);
      const int nt = tiles_of(len);
      const int te = static_cast<int>(min(static_cast<int64_t>(nt), t + (x1 - x)));
      const bool direct = t == 0 && te == nt;
      const int slot = (blockIdx.x * 2 + (t == 0 ? 1 : 0));
      bool first = true;
      if (t == 0 && te < nt && pt == 0) {
        // the group goes on in the ranges after this one, up to the one that holds its last tile
        const int64_t last = x + nt - 1;
        const int c1 = static_cast<int>(((last + 1) * parts - 1) / total);
        p.meta[blockIdx.x] = make_int4(g, c1 - part + 1, 0, 0);
      }
      const int32_t* list = PAGED ? p.block_table + static_cast<int64_t>(g) * p.max_blocks
                                  : p.slots + static_cast<int64_t>(g) * p.ld_slots;
      x += te - t;
      for (; t < te; ++t) {
        // ---- the tile's rows: slot of key `lane` and `lane + 32`, -1 where there is none
        int64_t sl[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int j = t * kAttnKeys + h * 32 + lane;
          int64_t v = -1;
          if (j < len) {
            if (PAGED) {
              const int pg = __ldg(list + t);  // a tile is a page
              if (pg >= 0 && pg < p.num_slots / kPageSize) v = static_cast<int64_t>(pg) * kPageSize + h * 32 + lane;
              else bad |= kStatusBadPage;
            } else {
              v = __ldg(list + j);
              if (v >= p.num_slots) {
                v = -1;
                bad |= kStatusBadSlot;
              }
            }
          }
          sl[h] = v;
        }
        const unsigned long long mask =
            __ballot_sync(0xFFFFFFFFu, sl[0] >= 0) |
            (static_cast<unsigned long long>(__ballot_sync(0xFFFFFFFFu, sl[1] >= 0)) << 32);
        const bool last = t == te - 1;
        const bool null = mask == 0;
        if (null && !last) continue;  // nothing to do and nothing to say
        const int st = i & 1;
        const uint32_t ph = (i >> 1) & 1;
        // ---- describe the tile.  The entry was tile i - 4's; the values of
        // tile i - 2 have begun, so every role is past tile i - 4.
        if (!warp_wait(&ms.empty[st][0], ph ^ 1, abort_flag, p.status, limit) ||
            !warp_wait(&ms.empty[st][4], ph ^ 1, abort_flag, p.status, limit)) {
          ok = false;
          break;
        }
        if (pt == 0) {
          Info& f = ms.info[i & (kInfo - 1)];
          f.mask = mask;
          f.flags = (first ? kFirst : 0) | (last ? kLast : 0) | (null ? kNull : 0) | (direct ? kDirect : 0);
          f.group = g;
          f.ends = PAGED ? len - p.R + 1 - t * kAttnKeys : 1 << 20;
          f.piece = slot;
          mbar_arrive(&ms.full[st][0]);
        }
        if (null) {
#pragma unroll
          for (int c = 0; c < kParts; ++c) {
            if (c > 0 && c < 4 && !warp_wait(&ms.empty[st][c], ph ^ 1, abort_flag, p.status, limit)) { ok = false; break; }
            mbar_arrive(&ms.full[st][c]);
          }
          if (!ok) break;
          ++i;
          continue;
        }
        if (first) {
          // ---- the group's query columns; free once the last tile's scores are done
          if (i > 0 && !warp_wait(&ms.empty[st ^ 1][4], ((i - 1) >> 1) & 1, abort_flag, p.status, limit)) {
            ok = false;
            break;
          }
          const int cols = p.R * p.H;
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int col = cg * kAttnCols + r0 + 16 * k;
            const bool v = col < cols;
            const int row = v ? col / p.H : 0, h = v ? col - row * p.H : 0;
            const uint8_t* src = reinterpret_cast<const uint8_t*>(
                p.q + (static_cast<int64_t>(g) * p.R + row) * p.q_row + h * p.q_head);
#pragma unroll
            for (int c = 0; c < kChunks; ++c)
              cp_async16(qdst0 + c * kChunkBytes + k * 2048, src + c * 128 + piece * 16, v ? 16 : 0);
          }
          cp_async_arrive(&ms.q_full);
        }
        // ---- the key rows
        const uint8_t* row[4];
        uint32_t n[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int64_t v = __shfl_sync(0xFFFFFFFFu, sl[k >> 1], (r0 + 16 * k) & 31);
          n[k] = v >= 0 ? 16 : 0;
          row[k] = p.kv + (v >= 0 ? v : 0) * (kLatentDim * 2) + piece * 16;
        }
        const uint32_t dst = dst0 + st * kStageBytes;
#pragma unroll
        for (int c = 0; c < kParts; ++c) {
          if (c > 0 && c < 4 && !warp_wait(&ms.empty[st][c], ph ^ 1, abort_flag, p.status, limit)) { ok = false; break; }
#pragma unroll
          for (int u = 0; u < (c < 4 ? 2 : 1); ++u) {
            const int ch = 2 * c + u;
#pragma unroll
            for (int k = 0; k < 4; ++k) cp_async16(dst + ch * kChunkBytes + k * 2048, row[k] + ch * 128, n[k]);
          }
          if (!(p.debug_withhold_first_tile && i == 0 && c == 0)) cp_async_arrive(&ms.full[st][c]);
        }
        if (!ok) break;
        first = false;
        ++i;
      }
    }
    // ---- the end of the stream
    if (ok) {
      const int st = i & 1;
      const uint32_t ph = (i >> 1) & 1;
      if (warp_wait(&ms.empty[st][0], ph ^ 1, abort_flag, p.status, limit)) {
        if (pt == 0) {
          ms.info[i & (kInfo - 1)].flags = kEnd;
          mbar_arrive(&ms.full[st][0]);
        }
        mbar_arrive(&ms.full[st][0]);
      }
    }
    cp_async_wait_all();
    if (bad && cg == 0) atomicOr(p.status, bad);
  } else if (warp == 8) {
    // ================================================================ MMA
    if (lane == 0) {
      constexpr uint32_t id_s = idesc_bf16_f32(64, 64, false), id_v = idesc_bf16_f32(128, 64, true);
      const uint32_t q_s = smem_u32(smem + kOffQ), k_s = smem_u32(smem + kOffK), p_s = smem_u32(smem + kOffP);
      int qi = 0, qg = 0, vi = 0, nq = 0;  // next tile and part for scores, next tile for values, query loads seen
      int qflags = 0;                      // flags of tile qi (known once its part 0 has landed)
      bool end = false;
      uint64_t t0 = global_timer_ns();
      uint32_t polls = 0;
      while (!(end && vi == qi)) {
        bool did = false;
        if (vi < qi && mbar_try_wait(&ms.p_full, vi & 1)) {
          // ---- values of tile vi
          const int st = vi & 1;
          const int f = ms.info[vi & (kInfo - 1)].flags;
          tc_fence_after();
          if (f & kNull) {
#pragma unroll
            for (int c = 0; c < 4; ++c) mbar_arrive(&ms.empty[st][c]);
            mbar_arrive(&ms.pv_done);
          } else {
#pragma unroll
            for (int c = 0; c < 4; ++c) {
#pragma unroll
              for (int ks = 0; ks < 4; ++ks)
                mma_bf16(tbase + kTmemO + c * 64,
                         smem_desc_mn_sw128(k_s + st * kStageBytes + 2 * c * kChunkBytes + ks * 2048),
                         smem_desc_k128_sw128(p_s + ks * 32), id_v, ks > 0 || !(f & kFirst));
              mma_commit(&ms.empty[st][c]);
            }
            mma_commit(&ms.pv_done);
          }
          ++vi;
          did = true;
        } else if (!end) {
          const int st = qi & 1;
          const uint32_t ph = (qi >> 1) & 1;
          if ((qg > 0 || mbar_try_wait(&ms.s_empty[st], ph ^ 1)) && mbar_try_wait(&ms.full[st][qg], ph)) {
            if (qg == 0) qflags = ms.info[qi & (kInfo - 1)].flags;
            if (qflags & kEnd) {
              mbar_arrive(&ms.s_full[st]);
              end = true;
            } else if (qflags & kNull) {
              if (++qg == kParts) {
                mbar_arrive(&ms.empty[st][4]);
                mbar_arrive(&ms.s_full[st]);
                ++qi;
                qg = 0;
              }
            } else {
              bool go = true;
              if (qg == 0 && (qflags & kFirst)) {
                go = wait_phase<kSpin>(&ms.q_full, nq & 1, abort_flag, p.status, limit);
                ++nq;
              }
              if (!go) break;
              fence_async_shared();
              tc_fence_after();
#pragma unroll 1
              for (int u = 0; u < (qg < 4 ? 2 : 1); ++u) {
                const int ch = 2 * qg + u;
#pragma unroll
                for (int ks = 0; ks < 4; ++ks)
                  mma_bf16(tbase + kTmemS + st * 64, smem_desc_k128_sw128(q_s + ch * kChunkBytes + ks * 32),
                           smem_desc_k128_sw128(k_s + st * kStageBytes + ch * kChunkBytes + ks * 32), id_s,
                           ch > 0 || ks > 0);
              }
              if (++qg == kParts) {
                mma_commit(&ms.empty[st][4]);
                mma_commit(&ms.s_full[st]);
                ++qi;
                qg = 0;
              }
            }
            did = true;
          }
        }
        if (did) {
          polls = 0;
        } else if ((++polls & 63) == 0) {
          if (polls == 64) t0 = global_timer_ns();
          if (*abort_flag) break;
          if (global_timer_ns() - t0 > limit) {
            *abort_flag = 1;
            atomicOr(p.status, kStatusWaitTimeout);
            break;
          }
        }
      }
      // every MMA issued has finished before shared memory and TMEM go away
      mma_commit(&ms.drain);
      const uint64_t td = global_timer_ns();
      while (!mbar_try_wait(&ms.drain, 0) && global_timer_ns() - td < 200000000ull) {
      }
    }
    __syncwarp();
  } else if (warp < 4) {
    // ================================================================ softmax and output
    const uint32_t lane_base = static_cast<uint32_t>(warp) << 21;  // TMEM lane 32 * warp
    const int rr = warp * 16 + (lane >> 2);  // this thread's columns (heads): rr and rr + 8
    const int cq = 2 * (lane & 3);           // its keys: 8 j + cq + {0, 1}
    const int cols = p.R * p.H;
    int trow[2];                             // row within the group of each column
#pragma unroll
    for (int h = 0; h < 2; ++h) trow[h] = PAGED ? min((cg * kAttnCols + rr + 8 * h) / p.H, p.R - 1) : 0;
    uint8_t* prow = smem + kOffP + rr * 128 + 2 * cq;
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
    for (int i = 0;; ++i) {
      const int b = i & 1;
      // a wait that gave up is carried to the votes below, so that all four
      // warps leave together
      bool dead = !warp_wait(&ms.s_full[b], (i >> 1) & 1, abort_flag, p.status, limit);
      tc_fence_after();
      const Info& f = ms.info[i & (kInfo - 1)];
      const int flags = dead ? kNull : f.flags;
      const bool end = flags & kEnd;
      if (flags & kFirst) {
        m[0] = m[1] = -INFINITY;
        l[0] = l[1] = 0.f;
      }
      uint32_t w[16];
      float fac[2] = {1.f, 1.f};
      bool grow = false;
      if (!(flags & (kNull | kEnd))) {
        uint32_t r[32];
        tmem_ld_16x64(tbase + kTmemS + b * 64 + lane_base, r);
        tmem_ld_wait();
        tc_fence_before();
        mbar_arrive(&ms.s_empty[b]);
        const unsigned long long mask = f.mask;
        const int ends = f.ends;
        float mx[2] = {-INFINITY, -INFINITY};
        const bool whole = mask == ~0ull && ends >= kAttnKeys;
        if (!whole) {
#pragma unroll
          for (int j = 0; j < 32; ++j) {
            const int key = 8 * (j >> 2) + cq + (j & 1), h = (j >> 1) & 1;
            const bool real = (mask >> key) & 1;
            const bool seen = real && key < ends + trow[h];
            if (PAGED && real && !seen && !(fabsf(__uint_as_float(r[j])) < INFINITY)) {
              // a key that this row must not see is not finite: 0 * value would
              // not be 0, so its values become 0 (rows that see it have a
              // score that is not finite, and keep it)
              uint8_t* krow = smem + kOffK + b * kStageBytes + key * 128;
              for (int c = 0; c < 8; ++c)
                for (int x = 0; x < 8; ++x)
                  *reinterpret_cast<uint4*>(krow + c * kChunkBytes + x * 16) = make_uint4(0, 0, 0, 0);
            }
            if (!seen) r[j] = 0xFF800000u;
          }
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          mx[0] = fmaxf(mx[0], fmaxf(__uint_as_float(r[4 * j]), __uint_as_float(r[4 * j + 1])));
          mx[1] = fmaxf(mx[1], fmaxf(__uint_as_float(r[4 * j + 2]), __uint_as_float(r[4 * j + 3])));
        }
        float neg[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          mx[h] = fmaxf(mx[h], __shfl_xor_sync(0xFFFFFFFFu, mx[h], 1));
          mx[h] = fmaxf(mx[h], __shfl_xor_sync(0xFFFFFFFFu, mx[h], 2));
          mx[h] *= p.scale_log2;
          if (flags & kFirst) {
            m[h] = mx[h];
          } else if (mx[h] > m[h] + kRescaleLog2) {
            fac[h] = ex2(m[h] - mx[h]);
            m[h] = mx[h];
            l[h] *= fac[h];
            grow = true;
          }
          neg[h] = m[h] == -INFINITY ? 0.f : -m[h];
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const float a = ex2(fmaf(__uint_as_float(r[4 * j + 2 * h]), p.scale_log2, neg[h]));
            const float c = ex2(fmaf(__uint_as_float(r[4 * j + 2 * h + 1]), p.scale_log2, neg[h]));
            l[h] += a + c;
            w[2 * j + h] = pack_bf16(a, c);
          }
        }
      } else if (!end && !dead) {
        mbar_arrive(&ms.s_empty[b]);
      }
      // the previous value product is done: the weights' buffer is free and the sums hold still
      if (i > 0 && !dead && !warp_wait(&ms.pv_done, (i - 1) & 1, abort_flag, p.status, limit)) dead = true;
      if (bar_red_or(1, kSoftmax, dead || end || grow)) {
        if (bar_red_or(1, kSoftmax, dead || end)) break;
        if ((lane & 3) == 0) {
          ms.stat_m[rr] = fac[0];
          ms.stat_m[rr + 8] = fac[1];
        }
        named_bar_sync(2, kSoftmax);
        tc_fence_after();
#pragma unroll 1
        for (int c = 0; c < 8; ++c) {
          uint32_t o[32];
          tmem_ld32(tbase + kTmemO + c * 32 + lane_base, o);
          tmem_ld_wait();
#pragma unroll
          for (int k = 0; k < 32; ++k)
            o[k] = __float_as_uint(__uint_as_float(o[k]) * ms.stat_m[(c & 1) * 32 + k]);
          tmem_st32(tbase + kTmemO + c * 32 + lane_base, o);
        }
        tmem_st_wait();
        named_bar_sync(2, kSoftmax);  // the factors are read before they are written again
      }
      if (!(flags & kNull)) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          *reinterpret_cast<uint32_t*>(prow + ((j ^ (rr & 7)) << 4)) = w[2 * j];
          *reinterpret_cast<uint32_t*>(prow + 8 * 128 + ((j ^ (rr & 7)) << 4)) = w[2 * j + 1];
        }
        fence_async_shared();
      }
      tc_fence_before();
      mbar_arrive(&ms.p_full);
      if (!(flags & kLast)) continue;

      // ---- the segment's end: its sums, divided (a whole group) or as they are (a cut one)
      const int group = f.group, slot = f.piece;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        l[h] += __shfl_xor_sync(0xFFFFFFFFu, l[h], 1);
        l[h] += __shfl_xor_sync(0xFFFFFFFFu, l[h], 2);
        if ((lane & 3) == 0) {
          ms.stat_m[rr + 8 * h] = m[h];
          ms.stat_l[rr + 8 * h] = l[h];
        }
      }
      const bool none = (flags & kNull) && (flags & kFirst);  // no key at all: the sums were never written
      const bool direct = flags & kDirect;
      if (!warp_wait(&ms.pv_done, i & 1, abort_flag, p.status, limit)) dead = true;
      if (bar_red_or(1, kSoftmax, dead)) break;
      tc_fence_after();
      const int n = min(kAttnCols, cols - cg * kAttnCols);
      const int64_t col0 = static_cast<int64_t>(group) * cols + cg * kAttnCols;
      if (tid < n) {
        const float mm = ms.stat_m[tid], ll = ms.stat_l[tid];
        if (!direct) p.part_ml[static_cast<int64_t>(slot) * kAttnCols + tid] = make_float2(mm, ll);
        else if (p.lse) p.lse[col0 + tid] = (mm + log2f(ll)) * 0.69314718055994531f;
      }
      named_bar_sync(2, kSoftmax);
      if (direct && tid < kAttnCols) {
        const float ll = ms.stat_l[tid];
        ms.stat_l[tid] = ll == 0.f ? 0.f : 1.f / ll;
      }
      named_bar_sync(2, kSoftmax);
      float* po = p.part_o + (static_cast<int64_t>(slot) * kAttnCols) * kLatent + warp * 32 + lane;
      uint16_t* oo = p.out + col0 * kLatent + warp * 32 + lane;
#pragma unroll 1
      for (int c = 0; c < 8; ++c) {  // 128 values c / 2, columns 32 (c % 2) + k
        if ((c & 1) * 32 >= n) continue;
        uint32_t o[32];
        if (none) {
#pragma unroll
          for (int k = 0; k < 32; ++k) o[k] = 0;
        } else {
          tmem_ld32(tbase + kTmemO + c * 32 + lane_base, o);
          tmem_ld_wait();
        }
#pragma unroll
        for (int k = 0; k < 32; ++k) {
          const int col = (c & 1) * 32 + k;
          if (col >= n) break;
          const float v = __uint_as_float(o[k]);
          if (direct)
            oo[static_cast<int64_t>(col) * kLatent + (c >> 1) * 128] =
                static_cast<uint16_t>(pack_bf16(v * ms.stat_l[col], 0.f));
          else
            po[static_cast<int64_t>(col) * kLatent + (c >> 1) * 128] = v;
        }
      }
      tc_fence_before();
      named_bar_sync(2, kSoftmax);  // stat_m and stat_l are read before the next group writes them
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 8) {
    tc_fence_after();
    tmem_dealloc(tbase, 512);
  }
}

// ---------------------------------------------------------------- joining cut groups

// Block (x, y): the group whose first piece CTA x holds, columns [8 y, 8 y + 8).
// The pieces lie in the CTAs x, x + ncg, ..., in key order: the first in its
// second slot, the others in their first.  128 threads take four values each.
constexpr int kJoinCols = 8;

__global__ void __launch_bounds__(128) latent_combine_kernel(const __grid_constant__ LatentAttnParams p) {
  griddep_wait();
  const int4 mt = p.meta[blockIdx.x];
  if (mt.y < 2) return;
  const int cols = p.R * p.H, cg = blockIdx.x % p.ncg;
  const int n = min(kAttnCols, cols - cg * kAttnCols);
  for (int col = blockIdx.y * kJoinCols; col < min(n, static_cast<int>(blockIdx.y + 1) * kJoinCols); ++col) {
    float top = -INFINITY;
    for (int k = 0; k < mt.y; ++k) {
      const int64_t slot = static_cast<int64_t>(blockIdx.x + k * p.ncg) * 2 + (k == 0 ? 1 : 0);
      top = fmaxf(top, __ldg(&p.part_ml[slot * kAttnCols + col].x));
    }
    const float ref = top == -INFINITY ? 0.f : top;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    float sum = 0.f;
    for (int k = 0; k < mt.y; ++k) {
      const int64_t slot = static_cast<int64_t>(blockIdx.x + k * p.ncg) * 2 + (k == 0 ? 1 : 0);
      const float2 ml = __ldg(&p.part_ml[slot * kAttnCols + col]);
      const float w = exp2f(ml.x - ref);
      const float4 v = __ldg(reinterpret_cast<const float4*>(p.part_o + (slot * kAttnCols + col) * kLatent) + threadIdx.x);
      sum = fmaf(ml.y, w, sum);
      acc.x = fmaf(v.x, w, acc.x);
      acc.y = fmaf(v.y, w, acc.y);
      acc.z = fmaf(v.z, w, acc.z);
      acc.w = fmaf(v.w, w, acc.w);
    }
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    const int64_t oc = static_cast<int64_t>(mt.x) * cols + cg * kAttnCols + col;
    reinterpret_cast<uint2*>(p.out + oc * kLatent)[threadIdx.x] =
        make_uint2(pack_bf16(acc.x * inv, acc.y * inv), pack_bf16(acc.z * inv, acc.w * inv));
    if (threadIdx.x == 0 && p.lse) p.lse[oc] = (top + log2f(sum)) * 0.69314718055994531f;
  }
}

cudaError_t launch_latent_attn(const LatentAttnParams& p, bool fp8, bool paged, cudaStream_t st) {
  if (fp8) return cudaErrorNotSupported;
  auto kern = paged ? latent_attn_kernel<true> : latent_attn_kernel<false>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes);
  if (e != cudaSuccess) return e;
  const int grid = p.parts * p.ncg;
  kern<<<grid, kThreads, kSmemBytes, st>>>(p);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(grid), kAttnCols / kJoinCols);
  cfg.blockDim = dim3(128);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, latent_combine_kernel, p);
}

}  // namespace fp8idx
