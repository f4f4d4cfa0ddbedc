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
// thread asks once, which answers sooner where the phase is over already (4096^3 59.4 us, 61.6 without; 512 x 4096 x 4096 12.7
// and 13.6), then sleeps in the barrier hardware, up to 100 us a try, and gives up after 2^17 of them.
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

// A warp's copies of COUNT scales (rows or groups first .. first + COUNT - 1 of a block, zeros from `limit` on) to `to` in the
// background; `from` is that of row `first`. `wide`: rows are neighbours on 16-byte boundaries in every block.
template <int COUNT>
__device__ __forceinline__ void copy_scales(uint32_t to, const float* from, const Scales& s, bool wide, int first, int limit,
                                            int lane) {
  if (wide) {
#pragma unroll
    for (int i = 0; i < COUNT; i += 128) {
      const int r = i + 4 * lane, left = limit - first - r;
      if (r < COUNT)
        asm volatile("cp.async.ca.shared.global [%0], [%1], 16, %2;" ::"r"(to + 4u * r), "l"(left > 0 ? from + r : s.p),
                     "r"(left >= 4 ? 16 : left > 0 ? 4 * left : 0)
                     : "memory");
    }
  } else {
    const float* at = from + lane * s.row;
#pragma unroll
    for (int i = 0; i < COUNT; i += 32, at += 32 * s.row) {
      const int r = i + lane;
      const bool in = first + r < limit;
      if (r < COUNT) cp_async_4(to + 4u * r, in ? at : s.p, in ? 4u : 0u);
    }
  }
}
inline bool wide_scales(const Scales& s) {
  return s.row == 1 && (reinterpret_cast<uintptr_t>(s.p) & 15u) == 0 && s.block % 4 == 0;
}

}  // namespace fp8
}  // namespace t2s
