// Suspended mbarrier waits, barriers between blocks and kernels, packed fp32 pairs.
#pragma once

#include <stdint.h>

#include "ptx.cuh"

namespace ira {

// For kernels launched with launch_dependent: nothing of the previous kernel's is
// read or overwritten before the wait is over; the next one may be set up from now on.
__device__ __forceinline__ void await_previous_kernel() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// All threads of all blocks of the cluster arrive, then wait; reads before the one
// are done before writes after the other.  (Not .aligned: a warp's threads may come one by
// one, as out of a loop with a trip count of each thread's own.)
__device__ __forceinline__ void cluster_arrive() {
  asm volatile("barrier.cluster.arrive.release;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
}

// mbarrier waits that let the hardware suspend the warp (up to kSuspendNs)
// until the phase completes, instead of polling.
constexpr uint32_t kSuspendNs = 20000;
__device__ __forceinline__ bool mbar_try_wait_s(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity), "r"(kSuspendNs)
      : "memory");
  return ok != 0;
}
__device__ __forceinline__ bool wait1(uint32_t bar, uint32_t parity, volatile int* abort) {
  if (mbar_try_wait_s(bar, parity)) return true;
  const unsigned long long t0 = globaltimer();
  for (;;) {
    if (mbar_try_wait_s(bar, parity)) return true;
    if (*abort) return false;
    if (globaltimer() - t0 > kWaitTimeoutNs) {
      *abort = 1;
      return false;
    }
  }
}
__device__ __forceinline__ bool waitw(uint32_t bar, uint32_t parity, volatile int* abort) {
  if (__all_sync(0xffffffffu, mbar_try_wait_s(bar, parity))) return true;
  const unsigned long long t0 = globaltimer();
  const bool leader = (threadIdx.x & 31) == 0;
  for (;;) {
    if (__all_sync(0xffffffffu, mbar_try_wait_s(bar, parity))) return true;
    int stop = 0;
    if (leader) {
      if (*abort) {
        stop = 1;
      } else if (globaltimer() - t0 > kWaitTimeoutNs) {
        *abort = 1;
        stop = 1;
      }
    }
    if (__shfl_sync(0xffffffffu, stop, 0)) return false;
  }
}

// Packed fp32 pairs (two lanes of one 64-bit register, .x in the low half):
// fma / add / mul on both halves in one instruction, rounding as two scalar ones.
__device__ __forceinline__ uint64_t f2_pack(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ void f2_unpack(uint64_t v, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ uint64_t f2_fma(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t f2_add(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint64_t f2_mul(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

}  // namespace ira
