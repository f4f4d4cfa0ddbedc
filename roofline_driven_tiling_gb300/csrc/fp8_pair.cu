// fp8_pair.cu -- products of 8-bit operands with a scale for each block of 128 of K, on pairs of SMs (tcgen05
// .cta_group::2, kind::f8f6f4).
//
// A persistent launch takes tiles of 256 rows x 64, 128 or 256 columns, each by a cluster of two CTAs: each
// stages its 128 rows of A and half of the rows of B, a block of 128 bytes of K per ring slot. A block's sums are
// started afresh in one of two TMEM accumulators, and eight warps per CTA take them out, multiply them by
// the block's scales and add them to FP32 sums in their registers (128 a thread for a 256-wide tile), while
// the other accumulator fills. So the scales may be any FP32 numbers, and the tensor cores' truncating additions never
// run longer than 128 products.
#include <cuda.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>
#include <cstring>

#include "fp8_device.cuh"
#include "t2s_device.cuh"
#include "t2s_tmap.h"
#include "tc_gemm.cuh"

namespace t2s {
namespace fp8 {
namespace {

using ff::pack2;

constexpr int kRows = 128;  // A rows of one CTA
constexpr int kStages = 6;
constexpr int kMaxN = 256;
constexpr int kABytes = kRows * kBlock;
constexpr int kBBytes = kMaxN / 2 * kBlock;
constexpr int kStageBytes = kABytes + kBBytes;
constexpr int kEpiWarps = 8;
constexpr int kThreads = 128 + 32 * kEpiWarps;
constexpr int kStagingBytes = 4096;  // of a warp: 32 x 32 outputs of 4 bytes, or two boxes of 2
constexpr int kSmemBytes = kStages * kStageBytes + 1024 + 1024 + kEpiWarps * kStagingBytes;
static_assert(kSmemBytes <= 227 * 1024, "shared memory of one CTA");
constexpr uint32_t kTmemCols = 512;

struct PairParams {
  CUtensorMap a, b, c;
  Scales sa, sb;
  void* C;
  int64_t ldc;
  int M, N, blocks, tiles_m, tiles_n;
  int c_tma;
  uint32_t idesc;
  unsigned* status;
};

// Byte offset of 16-byte chunk `c` of row `r` in a box of 32 rows of 64 (64-byte swizzle) or 128 bytes.
template <bool WIDE>
__device__ __forceinline__ uint32_t chunk_at(int r, int c) {
  return WIDE ? static_cast<uint32_t>(r) * 128u + (static_cast<uint32_t>(c ^ (r & 7)) << 4)
              : static_cast<uint32_t>(r) * 64u + (static_cast<uint32_t>(c ^ ((r >> 1) & 3)) << 4);
}

// A lane's row of 32 sums, rounded, into the warp's box.
template <int TYPE>
__device__ __forceinline__ void put_row(uint32_t box, int lane, const uint64_t* v) {
  if constexpr (TYPE == kF32) {
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      const float2 lo = ff::halves(v[2 * c]), hi = ff::halves(v[2 * c + 1]);
      st_shared_v4(box + chunk_at<true>(lane, c), __float_as_uint(lo.x), __float_as_uint(lo.y), __float_as_uint(hi.x),
                   __float_as_uint(hi.y));
    }
  } else {
    constexpr int kKind = TYPE == kBf16 ? ff::kBf16 : ff::kF16;
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      uint32_t w[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 f = ff::halves(v[4 * c + i]);
        w[i] = ff::pack_f32<kKind>(f.x, f.y);
      }
      st_shared_v4(box + chunk_at<false>(lane, c), w[0], w[1], w[2], w[3]);
    }
  }
}

// Stores a warp's 32 x 32 outputs at (m, n) from its box: by TMA, or a row per instruction where rows do not
// start on 16-byte boundaries.
template <int TYPE>
__device__ __forceinline__ void store_unit(const PairParams& p, uint32_t box, int m, int n, int lane) {
  if (p.c_tma) {
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) tma_store_2d(&p.c, box, n, m);
    return;
  }
  __syncwarp();
  const int rows = n + lane < p.N ? min(32, p.M - m) : 0;
  const int64_t first = static_cast<int64_t>(m) * p.ldc + n + lane;
#pragma unroll 8
  for (int r = 0; r < 32; ++r) {
    if constexpr (TYPE == kF32) {
      float v;
      asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(box + chunk_at<true>(r, lane >> 2) + (lane & 3) * 4));
      if (r < rows) static_cast<float*>(p.C)[first + r * p.ldc] = v;
    } else {
      uint16_t v;
      asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(box + chunk_at<false>(r, lane >> 3) + (lane & 7) * 2));
      if (r < rows) static_cast<uint16_t*>(p.C)[first + r * p.ldc] = v;
    }
  }
  __syncwarp();
}

// Roles: warps 0 and 2 copy A and B, warp 1 issues the MMAs (rank 0 only), warps 4..11 take the sums.
// full[s] / empty[s] per ring slot, acc_full[b] / acc_empty[b] per accumulator; a role that gives up a bounded wait
// records it and stops, and the others' own waits end the same way.
// UNITS: groups of 32 columns of each of the two warps of a row quarter. VECTOR: a scale for every row of B.
template <int TYPE, int UNITS, bool VECTOR>
__global__ void __launch_bounds__(kThreads, 1) fp8_pair_kernel(const __grid_constant__ PairParams p) {
  extern __shared__ uint8_t smem_raw[];
  constexpr int kBn = 2 * UNITS * kUnit;
  constexpr uint32_t kSlotBytes = kABytes + kBn / 2 * kBlock;
  const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
  const uint32_t bars = base + kStages * kStageBytes;
  auto full = [&](int s) { return bars + 8u * s; };
  auto empty = [&](int s) { return bars + 8u * (kStages + s); };
  const uint32_t acc_full = bars + 16u * kStages, acc_empty = acc_full + 16u, mma_done = acc_empty + 16u;
  const uint32_t slot = mma_done + 8u, staging = bars + 1024u;
  unsigned* const status = p.status;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = static_cast<int>(cluster_ctarank());
  const int tile0 = static_cast<int>(cluster_id_x()), tile_step = static_cast<int>(cluster_count_x());
  const int tiles = p.tiles_m * p.tiles_n, blocks = p.blocks;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(full(s), 1);
      mbar_init(empty(s), 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(acc_full + 8u * b, 1);
      mbar_init(acc_empty + 8u * b, 2 * kEpiWarps);
    }
    mbar_init(mma_done, 1);
    mbar_fence_init();
  }
  if (warp == 0 && ff::elect_one()) tma_prefetch_desc(&p.a);
  if (warp == 2 && ff::elect_one()) tma_prefetch_desc(&p.b);
  if (warp == 3) tc::tmem_alloc<2>(slot, kTmemCols);
  tc::tc_fence_before();
  __syncthreads();
  cluster_sync_all();  // the peer's copies and commits arrive on these barriers
  ff::wait_for_earlier_kernels();
  tc::tc_fence_after();
  uint32_t tmem;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(tmem) : "r"(slot) : "memory");

  if (warp < 4) {
    if (warp == 0 || warp == 2) {
      const bool is_a = warp == 0;
      ff::Ring ring(base + (is_a ? 0 : kABytes), kStageBytes, full(0), empty(0), kStages, kBlock);
      const uint32_t bar0 = tc::map_to_rank(full(0), 0);  // both CTAs' copies complete on rank 0's
      const uint32_t expect = is_a && rank == 0 ? 2 * kSlotBytes : 0u;
      const CUtensorMap* map = is_a ? &p.a : &p.b;
      bool ok = true;
      for (int t = tile0; ok && t < tiles; t += tile_step) {
        int m0, n0;
        tc::tile_origin(t, p.tiles_m, p.tiles_n, 2 * kRows, kBn, m0, n0);
        const int at = is_a ? m0 + rank * kRows : n0 + rank * (kBn / 2);
        ok = ring.copy(0, blocks, expect, bar0, status,
                       [&](uint32_t st, int k0, uint32_t bar) { tc::tma_load_2d_pair(st, map, k0, at, bar); });
      }
      // Every slot's copies have landed and been read before the CTA may go.
      if (ok) ring.copy(0, kStages, 0u, bar0, status, [](uint32_t, int, uint32_t) {});
    } else if (warp == 1 && rank == 0) {
      const ff::OperandForm form = ff::operand_form(true);
      int s = 0;
      uint32_t phase = 0, use = 0, st = base;
      bool ok = true;
      for (int t = tile0; ok && t < tiles; t += tile_step) {
#pragma unroll 1
        for (int kb = 0; kb < blocks; ++kb, ++use) {
          const uint32_t b = use & 1u;
          const uint64_t da = ff::with_address(form, st), db = ff::with_address(form, st + kABytes);
          ok = __all_sync(0xffffffffu, ff::wait_bounded(acc_empty + 8u * b, ((use >> 1) & 1u) ^ 1u, status) &&
                                           ff::wait_bounded(full(s), phase, status));
          if (!ok) break;
          tc::tc_fence_after();
          mma_block<2>(tmem + b * kMaxN, da, db, p.idesc);
          if (ff::elect_one()) {
            tc::mma_commit_pair(empty(s));
            tc::mma_commit_pair(acc_full + 8u * b);
          }
          __syncwarp();
          st += kStageBytes;
          if (++s == kStages) {
            s = 0;
            st = base;
            phase ^= 1u;
          }
        }
      }
      // Every MMA issued above ends before TMEM is released.
      if (ff::elect_one()) tc::mma_commit<2>(mma_done);
      __syncwarp();
      ff::wait_bounded(mma_done, 0u, status);
    }
  } else {
    const int e = warp - 4, q = warp & 3, half = e >> 2;
    const uint32_t box = staging + static_cast<uint32_t>(e) * kStagingBytes;
    const uint32_t rows_at = tmem + (static_cast<uint32_t>(32 * q) << 16) + static_cast<uint32_t>(half * UNITS * kUnit);
    uint32_t use = 0;
    bool ok = true;
    for (int t = tile0; ok && t < tiles; t += tile_step) {
      int m0, n0;
      tc::tile_origin(t, p.tiles_m, p.tiles_n, 2 * kRows, kBn, m0, n0);
      n0 += half * UNITS * kUnit;
      const int m = m0 + rank * kRows + 32 * q;
      const bool row_in = m + lane < p.M;
      const float* sa = p.sa.p + static_cast<int64_t>(row_in ? m + lane : 0) * p.sa.row;
      // Column scales: of this lane's column of each group (VECTOR), else of all the warp's columns, which lie
      // within one group of 128.
      constexpr int kScales = VECTOR ? UNITS : 1;
      const int n_lane = VECTOR ? n0 + lane : n0;
      const float* sb = p.sb.p + static_cast<int64_t>(VECTOR ? n_lane : n_lane / kBlock) * p.sb.row;
      uint64_t sum[UNITS][kUnit / 2];
#pragma unroll
      for (int u = 0; u < UNITS; ++u)
#pragma unroll
        for (int i = 0; i < kUnit / 2; ++i) sum[u][i] = 0;
      // The next block's scales are on their way while this one's sums are taken.
      float a_next = 0.0f, b_next[kScales] = {};
      auto fetch = [&](int kb) {
        if (kb >= blocks) return;
        if (row_in) a_next = sa[kb * p.sa.block];
#pragma unroll
        for (int u = 0; u < kScales; ++u)
          if (n_lane + u * kUnit < p.N) b_next[u] = sb[kb * p.sb.block + u * kUnit * p.sb.row];
      };
      fetch(0);
#pragma unroll 1
      for (int kb = 0; kb < blocks; ++kb, ++use) {
        const float a = a_next, f = a * b_next[0];
        if constexpr (VECTOR) {
          __syncwarp();
#pragma unroll
          for (int u = 0; u < UNITS; ++u)
            asm volatile("st.shared.f32 [%0], %1;" ::"r"(box + 4u * (u * kUnit + lane)), "f"(b_next[u]) : "memory");
          __syncwarp();
        }
        fetch(kb + 1);
        ok = __all_sync(0xffffffffu, ff::wait_bounded(acc_full + 8u * (use & 1u), (use >> 1) & 1u, status));
        if (!ok) break;
        tc::tc_fence_after();
        const uint32_t acc = rows_at + (use & 1u) * kMaxN;
        uint32_t part[2][16];
        load_columns16(acc, part[0]);
#pragma unroll
        for (int u = 0; u < 2 * UNITS; ++u) {
          uint32_t(&x)[16] = part[u & 1];
          uint64_t* to = sum[u / 2] + u % 2 * 8;
          wait_columns16(x);
          if (u + 1 < 2 * UNITS) {
            load_columns16(acc + (u + 1) * 16, part[(u + 1) & 1]);
          } else {
            tc::tc_fence_before();
            __syncwarp();
            if (lane == 0) ff::arrive_remote(tc::map_to_rank(acc_empty + 8u * (use & 1u), 0));
          }
          if constexpr (VECTOR) {
            const uint64_t row = ff::both(a);
#pragma unroll
            for (int i = 0; i < 8; i += 2) {
              uint64_t lo, hi;
              lds128_pairs(box + 4u * (u * 16 + 2 * i), lo, hi);
              to[i] = ff::fma2(ff::mul2(pack2(__uint_as_float(x[2 * i]), __uint_as_float(x[2 * i + 1])), lo), row, to[i]);
              to[i + 1] = ff::fma2(ff::mul2(pack2(__uint_as_float(x[2 * i + 2]), __uint_as_float(x[2 * i + 3])), hi), row,
                                   to[i + 1]);
            }
          } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
              to[i] = ff::fma2(pack2(__uint_as_float(x[2 * i]), __uint_as_float(x[2 * i + 1])), ff::both(f), to[i]);
          }
        }
      }
      if (!ok) break;
#pragma unroll
      for (int u = 0; u < UNITS; ++u) {
        if (m >= p.M || n0 + u * kUnit >= p.N) break;
        if (lane == 0) bulk_wait_read_all();
        __syncwarp();
        put_row<TYPE>(box, lane, sum[u]);
        store_unit<TYPE>(p, box, m, n0 + u * kUnit, lane);
      }
      if (VECTOR && lane == 0) bulk_wait_read_all();  // the scales of the next tile go to the same place
    }
    if (lane == 0) bulk_wait_all();  // the stores read this CTA's shared memory
  }

  tc::tc_fence_before();
  __syncthreads();
  cluster_sync_all();  // neither CTA goes while the other may use its memory, barriers or TMEM
  if (warp == 3) {
    tc::tc_fence_after();
    tc::tmem_dealloc<2>(tmem, kTmemCols);
  }
}

// Resident clusters of a kernel on the current device, looked up once.
template <int TYPE, int UNITS, bool VECTOR>
cudaError_t resident_clusters(int* out) {
  constexpr int kMaxDevices = 64;
  static std::atomic<int> known[kMaxDevices];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
  int n = known[dev].load(std::memory_order_acquire);
  if (n == 0) {
    auto kern = fp8_pair_kernel<TYPE, UNITS, VECTOR>;
    if ((e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes)) != cudaSuccess)
      return e;
    int sms = 0;
    if ((e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.gridDim = dim3(static_cast<unsigned>(sms / 2 * 2));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kSmemBytes;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if ((e = cudaOccupancyMaxActiveClusters(&n, kern, &cfg)) != cudaSuccess) return e;
    if (n < 1) return cudaErrorInvalidConfiguration;
    known[dev].store(n, std::memory_order_release);
  }
  *out = n;
  return cudaSuccess;
}

template <int TYPE, int UNITS, bool VECTOR>
cudaError_t launch(const ProductTask& t, cudaStream_t stream, unsigned* status) {
  constexpr int kBn = 2 * UNITS * kUnit;
  constexpr int kBytes = TYPE == kF32 ? 4 : 2;
  int resident = 0;
  cudaError_t e = resident_clusters<TYPE, UNITS, VECTOR>(&resident);
  if (e != cudaSuccess) return e;
  PairParams p;
  memset(&p, 0, sizeof(p));
  p.sa = t.sa, p.sb = t.sb;
  p.C = t.C, p.ldc = t.ldc;
  p.M = static_cast<int>(t.M), p.N = static_cast<int>(t.N);
  p.blocks = static_cast<int>(blocks_of(t.K));
  p.idesc = instruction(t.format_a, t.format_b, 2 * kRows, kBn);
  p.status = status;
  const int64_t tiles_m = (t.M + 2 * kRows - 1) / (2 * kRows), tiles_n = (t.N + kBn - 1) / kBn;
  if (tiles_m > 0x7fffffff / tiles_n) return cudaErrorInvalidConfiguration;
  p.tiles_m = static_cast<int>(tiles_m), p.tiles_n = static_cast<int>(tiles_n);
  if (p.blocks > 0) {
    if ((e = encode_tmap_8bit_2d(&p.a, t.A, t.K, t.M, t.lda, kBlock, kRows, CU_TENSOR_MAP_SWIZZLE_128B)) != cudaSuccess)
      return e;
    if ((e = encode_tmap_8bit_2d(&p.b, t.B, t.K, t.N, t.ldb, kBlock, kBn / 2, CU_TENSOR_MAP_SWIZZLE_128B)) != cudaSuccess)
      return e;
  }
  // Stores by TMA where rows lie on 16-byte boundaries and hold whole 16-byte words (a clipped store still
  // writes the whole of its last 16 bytes).
  p.c_tma = ((reinterpret_cast<uintptr_t>(t.C) | static_cast<uintptr_t>(t.ldc * kBytes) |
              static_cast<uintptr_t>(t.N * kBytes)) & 15u) == 0;
  if (p.c_tma) {
    e = TYPE == kF32 ? encode_tmap_f32_2d(&p.c, t.C, t.N, t.M, t.ldc, kUnit, 32, CU_TENSOR_MAP_SWIZZLE_128B)
                     : encode_tmap_16bit_2d(&p.c, t.C, t.N, t.M, t.ldc, kUnit, 32, CU_TENSOR_MAP_SWIZZLE_64B);
    if (e != cudaSuccess) return e;
  }
  const int64_t tiles = tiles_m * tiles_n;
  const ff::LaunchShape shape{dim3(static_cast<unsigned>(2 * (tiles < resident ? tiles : resident))), kThreads, 2, kSmemBytes};
  return ff::launch_early(stream, shape, fp8_pair_kernel<TYPE, UNITS, VECTOR>, p);
}

template <int TYPE, int UNITS>
cudaError_t launch_scales(const ProductTask& t, cudaStream_t stream, unsigned* status) {
  return t.b_group == 1 ? launch<TYPE, UNITS, true>(t, stream, status) : launch<TYPE, UNITS, false>(t, stream, status);
}

template <int TYPE>
cudaError_t launch_width(const ProductTask& t, int width, cudaStream_t stream, unsigned* status) {
  return width == 256 ? launch_scales<TYPE, 4>(t, stream, status)
                      : width == 128 ? launch_scales<TYPE, 2>(t, stream, status) : launch_scales<TYPE, 1>(t, stream, status);
}

}  // namespace

cudaError_t run_pair(const ProductTask& t, int width, cudaStream_t stream, unsigned* status) {
  return t.type == kF32 ? launch_width<kF32>(t, width, stream, status)
                        : t.type == kBf16 ? launch_width<kBf16>(t, width, stream, status)
                                          : launch_width<kF16>(t, width, stream, status);
}

}  // namespace fp8
}  // namespace t2s
