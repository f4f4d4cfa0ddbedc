// fp8_device.cuh -- device helpers of the 8-bit product kernels beside ff_device.cuh.
#pragma once

#include "ff_device.cuh"
#include "ff_math.cuh"
#include "fp8_internal.h"

namespace t2s {
namespace fp8 {


// The MMAs of one block of 128 values of K (four of K = 32) by one elected thread of a converged warp, from
// 128-byte swizzled K-major rows; D starts from the first product.
template <int G>
__device__ __forceinline__ void mma_block(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc) {
  if constexpr (G == 2) {
    asm volatile(
        "{\n\t.reg .pred e;\n\t.reg .b64 a, b;\n\t"
        "elect.sync _|e, 0xffffffff;\n\t"
        "@e tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, 0;\n\t"
        "add.u64 a, %1, 2;\n\tadd.u64 b, %2, 2;\n\t"
        "@e tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], a, b, %3, 1;\n\t"
        "add.u64 a, a, 2;\n\tadd.u64 b, b, 2;\n\t"
        "@e tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], a, b, %3, 1;\n\t"
        "add.u64 a, a, 2;\n\tadd.u64 b, b, 2;\n\t"
        "@e tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], a, b, %3, 1;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc)
        : "memory");
  } else {
    asm volatile(
        "{\n\t.reg .pred e;\n\t.reg .b64 a, b;\n\t"
        "elect.sync _|e, 0xffffffff;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, 0;\n\t"
        "add.u64 a, %1, 2;\n\tadd.u64 b, %2, 2;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a, b, %3, 1;\n\t"
        "add.u64 a, a, 2;\n\tadd.u64 b, b, 2;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a, b, %3, 1;\n\t"
        "add.u64 a, a, 2;\n\tadd.u64 b, b, 2;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a, b, %3, 1;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc)
        : "memory");
  }
}

__device__ __forceinline__ bool try_barrier(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}

// A bounded barrier wait without a call in it (a kernel that moves registers between its warps can make none): the
// thread asks once, which answers sooner where the phase is over already (4096^3 67 -> 65 us), then sleeps in the barrier
// hardware, up to 100 us a try, and gives up after 2^17 of them.
__device__ __forceinline__ bool wait_counted(uint32_t bar, uint32_t parity, unsigned* status) {
  if (try_barrier(bar, parity)) return true;
#pragma unroll 1
  for (int tries = 0; tries < 1 << 17; ++tries) {
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
  record_status(status, T2S_ERR_TIMEOUT);
  return false;
}

// Instruction descriptor: D FP32, the operands' formats, both K-major, N and M.
inline uint32_t instruction(int format_a, int format_b, int m, int n) {
  return (1u << 4) | (static_cast<uint32_t>(format_a) << 7) | (static_cast<uint32_t>(format_b) << 10) |
         (static_cast<uint32_t>(n >> 3) << 17) | (static_cast<uint32_t>(m >> 4) << 24);
}

// The scale of row (or group) r and block b.
__device__ __forceinline__ float scale_at(const Scales& s, int64_t r, int64_t b) { return s.p[r * s.row + b * s.block]; }

}  // namespace fp8
}  // namespace t2s
