// wait.cuh -- bounded mbarrier waits and the barrier vote, shared by the
// warp-specialised kernels.
#pragma once
#include <cstdint>

#include "kernels.cuh"
#include "ptx.cuh"

namespace fp8idx {

// Bounded wait on an mbarrier phase.  Gives up when another role has
// aborted or after `limit_ns`, flagging the device status; never traps.
// NAP_NS == 0 polls with try_wait (for the epilogue's own hand-offs, where
// the phase is normally complete already); NAP_NS > 0 passes try_wait a
// suspend-time hint of 16 NAP_NS, so the thread sleeps in hardware until the
// phase completes or the hint runs out, and a role that is ahead of the
// epilogue (MMA issue, TMA producer, idle select warps) takes few issue
// slots from it.  The abort flag and the clock are looked at every 8 tries.
template <uint32_t NAP_NS>
static __device__ __noinline__ bool wait_slow(uint64_t* bar, uint32_t parity, volatile int* abort_flag,
                                       int* status, unsigned long long limit_ns) {
  const uint64_t t0 = global_timer_ns();
  for (uint32_t it = 1;; ++it) {
    if (NAP_NS == 0 ? mbar_try_wait(bar, parity) : mbar_try_wait_hint(bar, parity, 16 * NAP_NS)) return true;
    if ((it & 7) == 0) {
      if (*abort_flag) return false;
      if (global_timer_ns() - t0 > limit_ns) {
        *abort_flag = 1;
        atomicOr(status, kStatusWaitTimeout);
        return false;
      }
    }
  }
}

// Nap lengths (ns) by role, the unit of each role's suspend-time hint: the
// epilogue polls; the MMA thread's is short (it has slack against the
// epilogue but must not delay the next tile); the producer runs stages
// ahead; idle roles sleep long.
#ifndef FP8IDX_NAP_MMA_NS
#define FP8IDX_NAP_MMA_NS 64
#endif
#ifndef FP8IDX_NAP_PRODUCER_NS
#define FP8IDX_NAP_PRODUCER_NS 256
#endif
#ifndef FP8IDX_NAP_IDLE_NS
#define FP8IDX_NAP_IDLE_NS 2048
#endif
constexpr uint32_t kSpin = 0, kNap = FP8IDX_NAP_MMA_NS, kProd = FP8IDX_NAP_PRODUCER_NS,
                   kSleep = FP8IDX_NAP_IDLE_NS;

template <uint32_t NAP_NS>
__device__ __forceinline__ bool wait_phase(uint64_t* bar, uint32_t parity, volatile int* abort_flag,
                                           int* status, unsigned long long limit_ns) {
  if (mbar_try_wait(bar, parity)) return true;
  return wait_slow<NAP_NS>(bar, parity, abort_flag, status, limit_ns);
}

// Uniform OR over the threads of a named barrier.
__device__ __forceinline__ bool bar_red_or(int id, int nthreads, bool pred) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %1, 0;\n\t"
      "bar.red.or.pred q, %2, %3, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(static_cast<uint32_t>(pred)), "r"(id), "r"(nthreads)
      : "memory");
  return r != 0;
}

}  // namespace fp8idx
