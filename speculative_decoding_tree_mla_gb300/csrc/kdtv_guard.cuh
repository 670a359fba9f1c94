// Bounded waits of the tensor-core kernels whose status is the caller's word.
#pragma once

#include "kdtv_ptx.cuh"

namespace kdtv {
namespace {

using namespace ptx;

struct Guard {
  volatile uint32_t* abort;      // shared memory
  unsigned int* status;
  uint32_t limit;                // ns, below 2^32
};
__device__ __forceinline__ uint32_t timer_lo() {
  uint32_t t;
  asm volatile("mov.u32 %0, %%globaltimer_lo;" : "=r"(t));
  return t;
}
// Short code: a wait stands at some thirty places of loops that share an
// instruction cache.
__device__ __forceinline__ bool wait(const Guard& g, uint32_t bar, uint32_t parity) {
  if (__builtin_expect(mbar_try_wait(bar, parity), 1)) return true;
  const uint32_t t0 = timer_lo();
#pragma unroll 1
  while (!mbar_try_wait_sleep(bar, parity, 20000u)) {
    if (*g.abort) return false;
    if (timer_lo() - t0 > g.limit) {
      atomicExch(g.status, (unsigned)KDTV_ERR_DEVICE_TIMEOUT);   // over any other code: the combine kernel asks
      *g.abort = 1u;
      return false;
    }
  }
  return true;
}
// The same by polling: for a single thread on the critical path, which would pay the wake-up from a sleep (a few
// hundred cycles) at every phase.
__device__ __forceinline__ bool wait_poll(const Guard& g, uint32_t bar, uint32_t parity) {
  if (__builtin_expect(mbar_test_wait(bar, parity), 1)) return true;
  const uint32_t t0 = timer_lo();
#pragma unroll 1
  for (uint32_t i = 1; !mbar_test_wait(bar, parity); ++i) {
    if (i & 63u) continue;
    if (*g.abort) return false;
    if (timer_lo() - t0 > g.limit) {
      atomicExch(g.status, (unsigned)KDTV_ERR_DEVICE_TIMEOUT);
      *g.abort = 1u;
      return false;
    }
  }
  return true;
}
// Waits for asynchronous work that is in flight and will finish (limited all the same).
__device__ __forceinline__ void drain(const Guard& g, uint32_t bar, uint32_t parity) {
  const uint32_t t0 = timer_lo();
#pragma unroll 1
  while (!mbar_try_wait(bar, parity))
    if (timer_lo() - t0 > g.limit) return;
}
__device__ __forceinline__ bool wait_warp(const Guard& g, uint32_t bar, uint32_t parity) {
  return __all_sync(0xffffffffu, wait(g, bar, parity));
}

}  // namespace
}  // namespace kdtv
