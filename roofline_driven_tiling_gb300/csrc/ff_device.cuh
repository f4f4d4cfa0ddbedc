// ff_device.cuh -- device helpers of the feed-forward kernels beside t2s_device.cuh.
#pragma once

#include "t2s_device.cuh"

namespace t2s {
namespace ff {

// The slow end of wait_bounded, out of the callers' loops.
static __device__ __noinline__ bool wait_long(uint32_t bar, uint32_t parity, unsigned* status) {
  return mbar_wait_bounded(bar, parity, status);
}

// A bounded barrier wait for loops whose round is a few hundred cycles: the thread sleeps in the
// barrier hardware (up to 100 us a try), and the limit's timer, whose read alone takes longer
// than such a round, is not touched before that has failed several times.
__device__ __forceinline__ bool wait_bounded(uint32_t bar, uint32_t parity, unsigned* status) {
#pragma unroll 1
  for (int tries = 0; tries < 64; ++tries) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity), "r"(100000u)
        : "memory");
    if (ok != 0) return true;
  }
  return wait_long(bar, parity, status);
}

}  // namespace ff
}  // namespace t2s
