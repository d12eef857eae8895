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

// Wait for phase `parity` of `bar`; false on abort or after `limit`.  lanes: those of the
// warp that wait together and get one answer, as instructions of the whole warp behind it
// want (near the limit one lane may still see the phase end that another gave up); 0: the
// calling lane alone.
__device__ __forceinline__ bool wait_bar(uint64_t *bar, uint32_t parity, volatile int *abort,
                                         unsigned *status, unsigned lanes = 0,
                                         uint64_t limit = kWaitLimitNs) {
  bool ok = ptx::mbar_try_wait(bar, parity);
  if (!ok) {
    const uint64_t t0 = ptx::globaltimer();
    for (uint32_t it = 1;; ++it) {
      ok = ptx::mbar_try_wait(bar, parity);
      if (ok) break;
      if ((it & 63) == 0) {
        if (*abort) break;
        if (ptx::globaltimer() - t0 > limit) {
          atomicCAS(status, 0u, (unsigned)FP8_ERR_TIMEOUT);
          *abort = 1;
          break;
        }
      }
    }
  }
  return lanes ? __all_sync(lanes, ok) : ok;
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
