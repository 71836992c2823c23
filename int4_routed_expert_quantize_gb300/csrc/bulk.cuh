// The plain bulk copy, without a cache policy, and a bounded wait that looks at the clock late.
#pragma once

#include "coli_device.cuh"

namespace coli {

// global -> shared, completing on `bar`; both 16-byte aligned, bytes a multiple of 16
__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(smem_addr(dst)),
               "l"(src), "r"(bytes), "r"(smem_addr(bar))
               : "memory");
}

// A bounded wait by a whole warp: every lane sees the phase, and the lanes are together afterwards.  Reading the global timer takes
// longer than most waits (a lane of a ring's reader waits some hundred cycles; the timer takes about a thousand), so the limit
// counts from the 16th try on.
__device__ __forceinline__ bool ring_wait(uint64_t* bar, uint32_t parity, volatile int* abort_flag, int* status) {
  bool ok = mbar_try_wait(bar, parity);
  if (!ok) {
    uint64_t t0 = 0;
#pragma unroll 1
    for (uint32_t it = 1; !*abort_flag; ++it) {
      if (mbar_try_wait(bar, parity)) {
        ok = true;
        break;
      }
      if (it < 16) continue;
      const uint64_t now = global_ns();
      if (it == 16) t0 = now;
      if (now - t0 > kWaitLimitNs) {
        *abort_flag = 1;
        atomicExch(status, COLI_ETIMEOUT);
      }
    }
  }
  return __all_sync(FULL, ok);
}

}  // namespace coli
