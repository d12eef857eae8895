// Bounded waits on mbarriers for warp-specialised kernels.  `status` is the
// translation unit's device status word, read through fp8_get_device_status.
#pragma once

#include <stdint.h>

#include "common.cuh"
#include "ptx.cuh"

namespace fp8lin {
namespace pipe {

constexpr uint64_t kWaitLimitNs = 2000000000ull;  // 2 s
constexpr uint64_t kDrainLimitNs = 100000000ull;  // 0.1 s

// Wait for phase `parity` of `bar`; false on abort or timeout.
__device__ __forceinline__ bool wait_bar(uint64_t *bar, uint32_t parity, volatile int *abort,
                                         unsigned *status) {
  if (ptx::mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = ptx::globaltimer();
  for (uint32_t it = 1;; ++it) {
    if (ptx::mbar_try_wait(bar, parity)) return true;
    if ((it & 63) == 0) {
      if (*abort) return false;
      if (ptx::globaltimer() - t0 > kWaitLimitNs) {
        atomicCAS(status, 0u, (unsigned)FP8_ERR_TIMEOUT);
        *abort = 1;
        return false;
      }
    }
  }
}

// Bounded wait that ignores the abort flag (used only to drain in-flight work).
__device__ __forceinline__ void drain_wait(uint64_t *bar, uint32_t parity, unsigned *status) {
  const uint64_t t0 = ptx::globaltimer();
  while (!ptx::mbar_try_wait(bar, parity))
    if (ptx::globaltimer() - t0 > kDrainLimitNs) {
      atomicCAS(status, 0u, (unsigned)FP8_ERR_TIMEOUT);
      return;
    }
}

}  // namespace pipe
}  // namespace fp8lin
