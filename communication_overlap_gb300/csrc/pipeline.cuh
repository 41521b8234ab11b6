// Bounded mbarrier waits of the expert layer's kernels, for rings of stages
// between warps that copy and warps that compute.
#pragma once

#include <cstdint>

#include "device_common.cuh"

namespace fo {
namespace tc {

constexpr uint64_t kWaitNs = 2000000000ull;   // 2 s per wait
constexpr uint64_t kDrainNs = 10000000ull;    // 10 ms while winding down

// Bounded wait for the phase with the given parity.  Gives up when another
// role aborted (shared flag) or after kWaitNs; then records the error.
static __device__ __noinline__ bool wait_slow(uint32_t bar, uint32_t parity,
                                              volatile int* abort_flag, int32_t* status) {
  // the clock is read only now and then: reading it costs more than most waits
  uint64_t t0 = 0;
  for (uint32_t i = 1;; ++i) {
    if (mbar_try_wait(bar, parity)) return true;
    if (i % 64) continue;
    if (*abort_flag) return false;
    const uint64_t now = globaltimer_ns();
    if (t0 == 0) t0 = now;
    if (now - t0 > kWaitNs) {
      *abort_flag = 1;
      atomicCAS(status, 0, int32_t(FO_ERR_TIMEOUT));
      return false;
    }
  }
}

// For a converged warp, whose lanes get one answer (what follows is often
// .aligned).
__device__ __forceinline__ bool wait_warp(uint32_t bar, uint32_t parity,
                                          volatile int* abort_flag, int32_t* status) {
  if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
  int ok = 0;
  if ((threadIdx.x & 31) == 0) ok = wait_slow(bar, parity, abort_flag, status);
  ok = __shfl_sync(0xffffffffu, ok, 0);
  __syncwarp();
  return ok != 0;
}

__device__ __forceinline__ uint64_t policy_evict_first() { return l2_evict_first(); }

__device__ __forceinline__ uint64_t policy_evict_last() {
  uint64_t pol;
  asm volatile("createpolicy.fractional.L2::evict_last.b64 %0, 1.0;" : "=l"(pol));
  return pol;
}

}  // namespace tc
}  // namespace fo
