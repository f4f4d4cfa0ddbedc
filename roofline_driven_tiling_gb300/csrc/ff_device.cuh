// ff_device.cuh -- device helpers of the feed-forward kernels beside t2s_device.cuh.
#pragma once

#include "ff_internal.h"
#include "t2s_device.cuh"
#include "t2s_tmap.h"

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

// A kernel launched by launch_early may start while the ones before it on its stream still run:
// what it does before wait_for_earlier_kernels touches no global memory. From then on the next kernel's
// start-up may overlap this one's work in the same way.
__device__ __forceinline__ void wait_for_earlier_kernels() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

struct LaunchShape {
  dim3 grid;
  int threads, cluster, smem;
};

template <class... P, class... A>
cudaError_t launch_early(cudaStream_t stream, const LaunchShape& shape, void (*kernel)(P...), const A&... args) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(shape.cluster);
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.gridDim = shape.grid;
  cfg.blockDim = dim3(static_cast<unsigned>(shape.threads));
  cfg.dynamicSmemBytes = static_cast<size_t>(shape.smem);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = shape.cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...);
}

constexpr int kBK = 64;                  // K block: 128-byte rows of 16-bit values
constexpr int kBoxBytes = 64 * kBK * 2;  // 64 outputs x 64 K rows of an MN-major operand

// A matrix descriptor without its address: K-major 128-byte-swizzled rows (8-row groups 1024
// bytes apart), or MN-major atoms (64 outputs x 8 K rows; the next 64 outputs one box further,
// the next 8 K rows 1024 bytes further). `step` is the advance of 16 K values.
struct OperandForm {
  uint64_t base;
  uint32_t step;
};
__device__ __forceinline__ OperandForm operand_form(bool k_major) {
  OperandForm f;
  f.base = (static_cast<uint64_t>(k_major ? 1 : kBoxBytes >> 4) << 16) | (static_cast<uint64_t>(1024 >> 4) << 32) |
           (static_cast<uint64_t>(1) << 46) | (static_cast<uint64_t>(2) << 61);
  f.step = (k_major ? 32 : 16 * 128) >> 4;
  return f;
}
__device__ __forceinline__ uint64_t with_address(const OperandForm& f, uint32_t addr) {
  return f.base | static_cast<uint64_t>((addr & 0x3ffffu) >> 4);
}

// The MMAs of one 64-deep K block (four of K = 16) by one elected thread of a converged warp:
// D (+)= A B^T from the descriptors `a` and `b`, which advance by the forms' steps; accumulate = 0
// starts D from the first product. Issued by a single diverged thread instead, the four took 264 cycles
// (every descriptor is moved to uniform registers), about as long as the widest ones compute.
template <int G>
__device__ __forceinline__ void mma_block(uint32_t d, uint64_t a, uint32_t a_step, uint64_t b, uint32_t b_step,
                                          uint32_t idesc, uint32_t accumulate) {
  if constexpr (G == 2) {
    asm volatile(
        "{\n\t.reg .pred e, p;\n\t.reg .b64 a, b, sa, sb;\n\t"
        "elect.sync _|e, 0xffffffff;\n\t"
        "setp.ne.b32 p, %6, 0;\n\t"
        "cvt.u64.u32 sa, %2;\n\tcvt.u64.u32 sb, %4;\n\t"
        "@e tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %3, %5, p;\n\t"
        "add.u64 a, %1, sa;\n\tadd.u64 b, %3, sb;\n\t"
        "@e tcgen05.mma.cta_group::2.kind::f16 [%0], a, b, %5, 1;\n\t"
        "add.u64 a, a, sa;\n\tadd.u64 b, b, sb;\n\t"
        "@e tcgen05.mma.cta_group::2.kind::f16 [%0], a, b, %5, 1;\n\t"
        "add.u64 a, a, sa;\n\tadd.u64 b, b, sb;\n\t"
        "@e tcgen05.mma.cta_group::2.kind::f16 [%0], a, b, %5, 1;\n\t}" ::"r"(d),
        "l"(a), "r"(a_step), "l"(b), "r"(b_step), "r"(idesc), "r"(accumulate)
        : "memory");
  } else {
    asm volatile(
        "{\n\t.reg .pred e, p;\n\t.reg .b64 a, b, sa, sb;\n\t"
        "elect.sync _|e, 0xffffffff;\n\t"
        "setp.ne.b32 p, %6, 0;\n\t"
        "cvt.u64.u32 sa, %2;\n\tcvt.u64.u32 sb, %4;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %3, %5, p;\n\t"
        "add.u64 a, %1, sa;\n\tadd.u64 b, %3, sb;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %5, 1;\n\t"
        "add.u64 a, a, sa;\n\tadd.u64 b, b, sb;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %5, 1;\n\t"
        "add.u64 a, a, sa;\n\tadd.u64 b, b, sb;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %5, 1;\n\t}" ::"r"(d),
        "l"(a), "r"(a_step), "l"(b), "r"(b_step), "r"(idesc), "r"(accumulate)
        : "memory");
  }
}

// Arrives on an mbarrier given by its shared::cluster address, possibly another CTA's. Ordered
// within the CTA only: for TMEM reads, which the tcgen05 fences order, not for memory (a release at cluster
// scope waits for every store in flight, about a microsecond).
__device__ __forceinline__ void arrive_remote(uint32_t cluster_addr) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}

// Starts reading 32 accumulator columns of the warp's 32 rows (one row per lane); the registers hold
// them after wait_columns, which stands between the load and every use.
__device__ __forceinline__ void load_columns(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, "
      "%11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, "
      "%28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]),
        "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]),
        "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]),
        "=r"(r[31])
      : "r"(taddr));
}
__device__ __forceinline__ void wait_columns(uint32_t (&r)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]),
                 "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]),
                 "+r"(r[13]), "+r"(r[14]), "+r"(r[15]), "+r"(r[16]), "+r"(r[17]), "+r"(r[18]),
                 "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]), "+r"(r[24]),
                 "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]), "+r"(r[30]),
                 "+r"(r[31])
               :
               : "memory");
}

// Writes 16 accumulator columns of the warp's 32 rows, and waits for all such writes of this warp.
__device__ __forceinline__ void store_columns16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, "
      "%11, %12, %13, %14, %15};" ::"r"(r[0]),
      "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
      "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void wait_stored_columns() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

// True in one lane of a converged warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t e;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(e));
  return e != 0;
}

// A copying warp's walk over a ring of shared-memory slots. The warp stays converged (its
// addresses and counters live in uniform registers); one elected lane announces and copies.
struct Ring {
  uint32_t first, stride, full, empty, slots;  // its part of slot 0, slot size, barriers of slot 0
  uint32_t st, s = 0, phase = 1;
  int depth;  // K values of a slot

  __device__ __forceinline__ Ring(uint32_t first_, uint32_t stride_, uint32_t full_, uint32_t empty_, uint32_t slots_,
                                  int depth_)
      : first(first_), stride(stride_), full(full_), empty(empty_), slots(slots_), st(first_), depth(depth_) {}

  // Slots of K [kb0, kb1), each into the next slot once that is free: issue(slot, k, barrier offset
  // from `bar0` by slot). `expect` bytes are announced on the slot's full barrier if not 0.
  template <class F>
  __device__ __forceinline__ bool copy(int kb0, int kb1, uint32_t expect, uint32_t bar0, unsigned* status, F&& issue) {
#pragma unroll 1
    for (int k0 = kb0 * depth; k0 < kb1 * depth; k0 += depth) {
      if (!__all_sync(0xffffffffu, wait_bounded(empty + 8u * s, phase, status))) return false;
      if (elect_one()) {
        if (expect != 0) mbar_arrive_expect_tx(full + 8u * s, expect);
        issue(st, k0, bar0 + 8u * s);
      }
      __syncwarp();
      st += stride;
      if (++s == slots) {
        s = 0;
        st = first;
        phase ^= 1u;
      }
    }
    return true;
  }
};

// The tensor map of an operand of `extent` x K values, in boxes of box_extent x 64 (K-major) or of
// 64 K rows x 64 (MN-major).
inline cudaError_t operand_map(CUtensorMap* m, const Operand& o, int64_t extent, int64_t K, uint32_t box_extent) {
  return o.k_major ? encode_tmap_16bit_2d(m, o.p, K, extent, o.ld, kBK, box_extent, CU_TENSOR_MAP_SWIZZLE_128B)
                   : encode_tmap_16bit_2d(m, o.p, extent, K, o.ld, 64, kBK, CU_TENSOR_MAP_SWIZZLE_128B);
}

}  // namespace ff
}  // namespace t2s
