// latent_store.cu -- new tokens into the paged latent cache (sm_100a).
//
// A token's cache entry is its latent vector c (512 values) and its key part
// k_pe (64 values) rotated by the token's position; the queries' rotary part
// is rotated by the same angles in the same launch.  For pair i < 32 of a
// 64-value vector x at position n, with (cos, sin) = cos_sin[n][i], [n][32+i]:
//   (a, b) = (x[2i], x[2i+1])  interleaved, or (x[i], x[32+i])  by halves
//   a' = a cos - b sin,  b' = b cos + a sin          (fp32, one rounding to bf16)
// The latent is stored as it is (bf16 pool), or as e4m3 codes with the
// indexer pool's rule s = max(max |c|, 1e-4) / 448, codes e4m3(c / s), the
// scale and the quotient in fp32 (a latent that holds a NaN has the scale NaN).
//
// One warp per (token, part): part 0 is the cache entry, part 1 + g the
// heads [16 g, 16 g + 16).  A vector of 64 values takes four lanes, eight
// pairs each, so a lane's eight cosines and sines are loaded once for all
// heads of the warp; all of a warp's loads are issued before any arithmetic.
// A plain HBM stream without reuse: 8192 tokens with 64 heads into an fp8 pool
// (151 MB) take 30.3 us, 5.0 TB/s, in a graph of 20 calls and 33.7 us, 4.5 TB/s,
// a call after another; 256 tokens with 16 heads 1.9 us in a graph, a launch.
// The large case is bound by DRAM's 128-byte runs (a head's rotary part lies
// 384 bytes from the next, its place in the queries 1152): 2 or 8 warps a CTA,
// and loads before the checks of position and slot, all take 30.3 us too.
#include <cstdint>

#include "kernels.cuh"
#include "latent.cuh"

namespace fp8idx {

namespace {

constexpr int kStoreWarps = 4;      // warps (tokens) per CTA
constexpr int kStoreHeads = 16;     // heads per warp, two passes of eight

__device__ __forceinline__ float bf_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// bf16 pair of (lo, hi), each rounded to nearest even.
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

__device__ __forceinline__ uint32_t e4m3x4_rn_sat(float a, float b, float c, float d) {
  uint16_t lo, hi;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
  return lo | (static_cast<uint32_t>(hi) << 16);
}

// |x| as bits: they order like the values, with NaN above infinity.
__device__ __forceinline__ uint32_t abs_bits(float f) { return __float_as_uint(f) & 0x7FFFFFFFu; }

struct Angles {
  float c[8], s[8];
};

__device__ __forceinline__ Angles load_angles(const float* __restrict__ row, int quarter) {
  Angles a;
  const float4* pc = reinterpret_cast<const float4*>(row) + 2 * quarter;
  const float4* ps = pc + 8;
  const float4 c0 = __ldg(pc), c1 = __ldg(pc + 1), s0 = __ldg(ps), s1 = __ldg(ps + 1);
  a.c[0] = c0.x; a.c[1] = c0.y; a.c[2] = c0.z; a.c[3] = c0.w;
  a.c[4] = c1.x; a.c[5] = c1.y; a.c[6] = c1.z; a.c[7] = c1.w;
  a.s[0] = s0.x; a.s[1] = s0.y; a.s[2] = s0.z; a.s[3] = s0.w;
  a.s[4] = s1.x; a.s[5] = s1.y; a.s[6] = s1.z; a.s[7] = s1.w;
  return a;
}

// Offsets (in 8-element units) of a lane's two 16-byte pieces of a 64-value
// vector: adjacent pieces (interleaved pairs) or the same piece of both halves.
template <bool INTER>
__device__ __forceinline__ int piece(int quarter, int k) {
  return INTER ? 2 * quarter + k : quarter + 4 * k;
}

template <bool INTER>
__device__ __forceinline__ void rotate8(uint4& x, uint4& y, const Angles& g) {
  uint32_t* X = &x.x;
  uint32_t* Y = &y.x;
  if (INTER) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float a = bf_lo(X[i]), b = bf_hi(X[i]);
      X[i] = pack_bf16(a * g.c[i] - b * g.s[i], b * g.c[i] + a * g.s[i]);
      const float e = bf_lo(Y[i]), f = bf_hi(Y[i]);
      Y[i] = pack_bf16(e * g.c[4 + i] - f * g.s[4 + i], f * g.c[4 + i] + e * g.s[4 + i]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float a0 = bf_lo(X[i]), a1 = bf_hi(X[i]), b0 = bf_lo(Y[i]), b1 = bf_hi(Y[i]);
      const float c0 = g.c[2 * i], c1 = g.c[2 * i + 1], s0 = g.s[2 * i], s1 = g.s[2 * i + 1];
      X[i] = pack_bf16(a0 * c0 - b0 * s0, a1 * c1 - b1 * s1);
      Y[i] = pack_bf16(b0 * c0 + a0 * s0, b1 * c1 + a1 * s1);
    }
  }
}

template <bool INTER, bool FP8>
__global__ void __launch_bounds__(kStoreWarps * 32) latent_store_kernel(const LatentStoreParams p) {
  const int64_t t = static_cast<int64_t>(blockIdx.x) * kStoreWarps + (threadIdx.x >> 5);
  if (t >= p.T) return;
  const int lane = threadIdx.x & 31, quarter = lane & 3;
  const int64_t pos = __ldg(p.positions + t);
  const bool in_table = pos >= 0 && pos < p.max_pos;  // else nothing of the token is written

  if (blockIdx.y > 0) {
    // ---- heads [h0, h0 + 16): eight a pass, four lanes a head
    const int h0 = (blockIdx.y - 1) * kStoreHeads + (lane >> 2);
    uint4 x[2], y[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int h = h0 + 8 * k;
      if (h < p.H) {
        const uint4* src = reinterpret_cast<const uint4*>(p.q_pe + t * p.q_row + h * p.q_head);
        x[k] = __ldg(src + piece<INTER>(quarter, 0));
        y[k] = __ldg(src + piece<INTER>(quarter, 1));
      }
    }
    if (!in_table) return;
    const Angles g = load_angles(p.cos_sin + pos * kRope, quarter);
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int h = h0 + 8 * k;
      if (h < p.H) {
        rotate8<INTER>(x[k], y[k], g);
        uint4* dst = reinterpret_cast<uint4*>(p.q_out + t * p.o_row + h * p.o_head);
        dst[piece<INTER>(quarter, 0)] = x[k];
        dst[piece<INTER>(quarter, 1)] = y[k];
      }
    }
    return;
  }

  // ---- the cache entry
  const int64_t sl = __ldg(p.slot + t);
  if (!in_table || sl < 0 || sl >= p.num_slots) return;
  const uint4* cs = reinterpret_cast<const uint4*>(p.c + t * p.c_ld);
  uint4 v[2], x, y;
  // bf16: 16-byte pieces lane and lane + 32; fp8: pieces 2 lane and 2 lane + 1, whose 16 codes are one store
  v[0] = __ldg(cs + (FP8 ? 2 * lane : lane));
  v[1] = __ldg(cs + (FP8 ? 2 * lane + 1 : lane + 32));
  if (lane < 4) {
    const uint4* src = reinterpret_cast<const uint4*>(p.k_pe + t * p.pe_ld);
    x = __ldg(src + piece<INTER>(quarter, 0));
    y = __ldg(src + piece<INTER>(quarter, 1));
    const Angles g = load_angles(p.cos_sin + pos * kRope, quarter);
    rotate8<INTER>(x, y, g);
    uint4* dst = reinterpret_cast<uint4*>(FP8 ? p.pe + sl * kRope : p.kv + sl * kLatentDim + kLatent);
    dst[piece<INTER>(quarter, 0)] = x;
    dst[piece<INTER>(quarter, 1)] = y;
  }
  if (!FP8) {
    uint4* dst = reinterpret_cast<uint4*>(p.kv + sl * kLatentDim);
    dst[lane] = v[0];
    dst[lane + 32] = v[1];
  } else {
    float f[16];
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t w = (&v[i >> 2].x)[i & 3];
      f[2 * i] = bf_lo(w);
      f[2 * i + 1] = bf_hi(w);
      m = max(m, max(abs_bits(f[2 * i]), abs_bits(f[2 * i + 1])));
    }
    m = __reduce_max_sync(0xFFFFFFFFu, m);
    // a latent with a NaN gets the scale NaN, so that attention to it is NaN
    const float sc = m > 0x7F800000u ? __uint_as_float(0x7FC00000u) : fmaxf(__uint_as_float(m), 1e-4f) / 448.0f;
    uint4 o;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      (&o.x)[i] = e4m3x4_rn_sat(f[4 * i] / sc, f[4 * i + 1] / sc, f[4 * i + 2] / sc, f[4 * i + 3] / sc);
    reinterpret_cast<uint4*>(p.codes + sl * kLatent)[lane] = o;
    if (lane == 0) p.scales[sl] = sc;
  }
}

}  // namespace

cudaError_t launch_latent_store(const LatentStoreParams& p, bool interleaved, cudaStream_t st) {
  const dim3 grid(static_cast<unsigned>((p.T + kStoreWarps - 1) / kStoreWarps),
                  static_cast<unsigned>(1 + (p.q_pe ? (p.H + kStoreHeads - 1) / kStoreHeads : 0)));
  const dim3 block(kStoreWarps * 32);
  const bool fp8 = p.codes != nullptr;
  if (interleaved && fp8) latent_store_kernel<true, true><<<grid, block, 0, st>>>(p);
  else if (interleaved) latent_store_kernel<true, false><<<grid, block, 0, st>>>(p);
  else if (fp8) latent_store_kernel<false, true><<<grid, block, 0, st>>>(p);
  else latent_store_kernel<false, false><<<grid, block, 0, st>>>(p);
  return cudaGetLastError();
}

}  // namespace fp8idx
