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

// mbar_try_wait that may sleep up to 20 us for the phase
__device__ __forceinline__ bool mbar_sleep_wait(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, 20000;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_addr(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}

// A bounded wait by a whole warp: every lane sees the phase, and the lanes are together afterwards.  A waiting warp sleeps and takes no
// issue slots from the working ones; the limit counts from the second try on.
__device__ __forceinline__ bool ring_wait(uint64_t* bar, uint32_t parity, volatile int* abort_flag, int* status) {
  bool ok = mbar_sleep_wait(bar, parity);
  if (!ok) {
    const uint64_t t0 = global_ns();
#pragma unroll 1
    while (!*abort_flag) {
      if (mbar_sleep_wait(bar, parity)) {
        ok = true;
        break;
      }
      if (global_ns() - t0 > kWaitLimitNs) {
        *abort_flag = 1;
        atomicExch(status, COLI_ETIMEOUT);
      }
    }
  }
  return __all_sync(FULL, ok);
}

}  // namespace coli
