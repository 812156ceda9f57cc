// Waits on mbarriers that end in any case: on expiry the status word latches
// an error and the block's other roles are told to stop.
#pragma once
#include <cstdint>

#include "ptx.cuh"

namespace tpf {

// Status word bits (workspace word 0).
constexpr uint32_t ST_TIMEOUT = 1u;

// Bounded wait; false on timeout (latched) or when another role aborted.
__device__ __forceinline__ bool wait_bar(uint32_t bar, uint32_t parity, uint64_t timeout_ns, uint32_t* status,
                                         volatile int32_t* abort_flag, uint32_t role) {
  if (mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = globaltimer_ns();
  uint32_t n = 0;
  while (true) {
    if (mbar_try_wait(bar, parity)) return true;
    if ((++n & 127u) == 0) {
      if (*abort_flag) return false;
      if (globaltimer_ns() - t0 > timeout_ns) {
        *abort_flag = 1;
        atomicOr(status, ST_TIMEOUT | (role << 4));
        return false;
      }
    }
  }
}

// Bounded wait used while shutting down: never latches, never aborts others.
__device__ __forceinline__ void drain_wait(uint32_t bar, uint32_t parity, uint64_t limit_ns) {
  const uint64_t t0 = globaltimer_ns();
  while (!mbar_try_wait(bar, parity)) {
    if (globaltimer_ns() - t0 > limit_ns) return;
  }
}

}  // namespace tpf
