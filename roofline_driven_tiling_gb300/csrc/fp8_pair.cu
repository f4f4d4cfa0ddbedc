// fp8_pair.cu -- products of 8-bit operands with a scale for each block of 128 of K, on pairs of SMs (tcgen05
// .cta_group::2, kind::f8f6f4).
//
// A persistent launch takes tiles of 256 rows x 64, 128 or 256 columns, each by a cluster of two CTAs: each
// stages its 128 rows of A and half of the rows of B, a block of 128 bytes of K per ring slot. A block's sums are
// started afresh in one of the TMEM accumulators (two of 256 columns, four of 128 or 64), and eight warps
// per CTA take them out, multiply them by the block's scales and add them to FP32 sums in their registers (128 a
// thread for a 256-wide tile), while the other accumulators fill. A warp of its own brings the scales to shared
// memory some blocks ahead: fetched by the sums' warps one block ahead, they held every block up for an L2 latency
// (0.49 us a block whatever its width). So the scales need be no powers of two, and the tensor cores' truncating additions never
// run longer than 128 products.
//
// Measured: 4096^3 59.5 us (2.3 PFLOP/s; copies and MMAs alone 41), with a scale for every column 87; 4096 x 8192 x 2048
// with those 86. The sums' warps bound it: a block of 256 columns takes the MMAs 0.3 us and them 0.40 (TMEM loads and
// one FMA a value), with a scale for every column, and so two operations a value, 0.62. Slower: 16 sums' warps and a ring
// slot less (4096^3 74 us), two chunks of TMEM loads under way (60.1; 101 with scales for every column), one accumulator
// for half of the columns.
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
constexpr int kRingBytes = 6 * 32768;
constexpr int kMaxN = 256;
constexpr int kABytes = kRows * kBlock;
constexpr int kMaxStages = 9;
constexpr int kEpiWarps = 8;
constexpr int kThreads = 128 + 32 * kEpiWarps;
constexpr int kChunk = 32;            // accumulator columns that a warp takes at a time
constexpr int kStagingBytes = 2048;   // of a warp: 32 rows of 64 bytes
constexpr int kScaleBlocks = 4;       // blocks whose scales come to shared memory together
constexpr int kScaleSlots = 2;
constexpr int kBlockScales = (kRows + kMaxN) * 4;  // of one block: its rows', its columns'
constexpr int kScaleBytes = kScaleBlocks * kBlockScales;
constexpr int kMaxBuffers = 4;
constexpr int kSmemBytes = kRingBytes + 1024 + 1024 + kEpiWarps * kStagingBytes + kScaleSlots * kScaleBytes;
static_assert(kSmemBytes <= 227 * 1024, "shared memory of one CTA");
constexpr uint32_t kTmemCols = 512;
// Registers: the block is launched with 168 a thread; the sums' warps take 224 and the others keep 56.
constexpr int kSumRegs = 224, kOtherRegs = 56;
static_assert(128 * kOtherRegs + 32 * kEpiWarps * kSumRegs <= kThreads * 168, "the launch's registers");

struct PairParams {
  CUtensorMap a, b, c;
  Scales sa, sb;
  void* C;
  int64_t ldc;
  int M, N, blocks, tiles_m, tiles_n;
  int c_tma, sa_wide, sb_wide;
  uint32_t idesc;
  unsigned* status;
};

// The columns of a warp's box of outputs (32 rows): 64 bytes.
template <int TYPE>
constexpr int box_columns() {
  return TYPE == kF32 ? 16 : 32;
}
// Byte offset of 16-byte word `c` of row `r` in a box (64-byte swizzle).
__device__ __forceinline__ uint32_t word_at(int r, int c) {
  return static_cast<uint32_t>(r) * 64u + (static_cast<uint32_t>(c ^ ((r >> 1) & 3)) << 4);
}

// A lane's row of a box of sums, rounded, into the box.
template <int TYPE>
__device__ __forceinline__ void put_row(uint32_t box, int lane, const uint64_t* v) {
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    uint32_t w[4];
    if constexpr (TYPE == kF32) {
      const float2 lo = ff::halves(v[2 * c]), hi = ff::halves(v[2 * c + 1]);
      w[0] = __float_as_uint(lo.x), w[1] = __float_as_uint(lo.y), w[2] = __float_as_uint(hi.x), w[3] = __float_as_uint(hi.y);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 f = ff::halves(v[4 * c + i]);
        w[i] = ff::pack_f32<TYPE == kBf16 ? ff::kBf16 : ff::kF16>(f.x, f.y);
      }
    }
    st_shared_v4(box + word_at(lane, c), w[0], w[1], w[2], w[3]);
  }
}

// Stores a warp's box of outputs at (m, n): by TMA, or one or two rows per instruction where rows do not start on
// 16-byte boundaries.
template <int TYPE>
__device__ __forceinline__ void store_box(const PairParams& p, uint32_t box, int m, int n, int lane) {
  constexpr int kColumns = box_columns<TYPE>(), kSize = TYPE == kF32 ? 4 : 2, kRowsAtOnce = 32 / kColumns;
  if (p.c_tma) {
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) tma_store_2d(&p.c, box, n, m);
    return;
  }
  __syncwarp();
  const int r0 = lane / kColumns, col = lane % kColumns, rows = n + col < p.N ? min(32, p.M - m) : 0;
  const int64_t first = static_cast<int64_t>(m) * p.ldc + n + col;
#pragma unroll 8
  for (int r = r0; r < 32; r += kRowsAtOnce) {
    const uint32_t from = box + word_at(r, col * kSize / 16) + col * kSize % 16;
    if constexpr (TYPE == kF32) {
      float v;
      asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(from));
      if (r < rows) static_cast<float*>(p.C)[first + r * p.ldc] = v;
    } else {
      uint16_t v;
      asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(from));
      if (r < rows) static_cast<uint16_t*>(p.C)[first + r * p.ldc] = v;
    }
  }
  __syncwarp();
}

// Roles: warp 0 copies A and B, warps 1 and 2 issue the MMAs (rank 0 only), warps 4..11 take the sums.
// Warp 3 holds TMEM and copies scales. full[s] / empty[s] per ring slot (empty also says that the slot's sums are in
// TMEM: one commit for both), acc_empty[b] per accumulator, scale_full[s] / scale_empty[s] per slot of scales; a role
// that gives up a bounded wait records it and stops, and the others' own waits end the same way.
// CHUNKS: groups of 32 columns of each of the two warps of a row quarter. VECTOR: a scale for every row of B.
template <int TYPE, int CHUNKS, bool VECTOR>
__global__ void __launch_bounds__(kThreads, 1) fp8_pair_kernel(const __grid_constant__ PairParams p) {
  extern __shared__ uint8_t smem_raw[];
  constexpr int kWarpN = CHUNKS * kChunk, kBn = 2 * kWarpN;
  constexpr uint32_t kSlotBytes = kABytes + kBn / 2 * kBlock;
  constexpr int kStages = kRingBytes / kSlotBytes;  // ring slots: six of a 256-wide tile's blocks, eight, nine
  static_assert(kStages <= kMaxStages, "barriers");
  const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
  const uint32_t bars = base + kRingBytes;
  auto full = [&](int s) { return bars + 8u * s; };
  auto empty = [&](int s) { return bars + 8u * (kMaxStages + s); };
  // At most as many accumulators as ring slots, so that empty[s] says for one block at a time that its sums are there.
  constexpr uint32_t kBuffers = kTmemCols / kBn < 4 ? kTmemCols / kBn : 4;
  static_assert(kBuffers <= kStages, "one commit for the slot and the sums");
  const uint32_t acc_empty = bars + 16u * kMaxStages;
  const uint32_t scale_full = acc_empty + 8u * kMaxBuffers, scale_empty = scale_full + 8u * kScaleSlots;
  const uint32_t mma_done = scale_empty + 8u * kScaleSlots, slot = mma_done + 8u;
  const uint32_t staging = bars + 1024u, scales = staging + kEpiWarps * kStagingBytes;
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
    for (uint32_t b = 0; b < kBuffers; ++b) mbar_init(acc_empty + 8u * b, 2 * kEpiWarps);
    for (int b = 0; b < kScaleSlots; ++b) {
      mbar_init(scale_full + 8u * b, 32);
      mbar_init(scale_empty + 8u * b, kEpiWarps);
    }
    mbar_init(mma_done, 2);
    mbar_fence_init();
  }
  if (warp == 0 && ff::elect_one()) tma_prefetch_desc(&p.a);
  if (warp == 1 && ff::elect_one()) tma_prefetch_desc(&p.b);
  if (warp == 3) tc::tmem_alloc<2>(slot, kTmemCols);
  tc::tc_fence_before();
  __syncthreads();
  cluster_sync_all();  // the peer's copies and commits arrive on these barriers
  ff::wait_for_earlier_kernels();
  tc::tc_fence_after();
  uint32_t tmem;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(tmem) : "r"(slot) : "memory");

  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
    // Ring slots one after another, `step` at a time.
    int s = warp == 2 ? 1 : 0;
    uint32_t phase = 0;
    auto next = [&](int step) {
      if ((s += step) >= kStages) {
        s -= kStages;
        phase ^= 1u;
      }
    };
    bool ok = true;
    if (warp == 0) {
      // The warp stays converged (its addresses and counters live in uniform registers); one elected lane announces and copies.
      const uint32_t full0 = tc::map_to_rank(full(0), 0);  // both CTAs' copies complete on rank 0's
      for (int t = tile0; ok && t < tiles; t += tile_step) {
        int m0, n0;
        tc::tile_origin(t, p.tiles_m, p.tiles_n, 2 * kRows, kBn, m0, n0);
        m0 += rank * kRows, n0 += rank * (kBn / 2);
#pragma unroll 1
        for (int kb = 0; kb < blocks; ++kb) {
          ok = __all_sync(0xffffffffu, wait_counted(empty(s), phase ^ 1u, status));
          if (!ok) break;
          if (ff::elect_one()) {
            const uint32_t st = base + static_cast<uint32_t>(s) * kSlotBytes;
            if (rank == 0) mbar_arrive_expect_tx(full(s), 2 * kSlotBytes);
            tc::tma_load_2d_pair(st, &p.a, kb * kBlock, m0, full0 + 8u * s);
            tc::tma_load_2d_pair(st + kABytes, &p.b, kb * kBlock, n0, full0 + 8u * s);
          }
          __syncwarp();
          next(1);
        }
      }
      // Every slot's copies have landed and been read before the CTA may go.
      for (int i = 0; ok && i < kStages; ++i) {
        ok = __all_sync(0xffffffffu, wait_counted(empty(s), phase ^ 1u, status));
        next(1);
      }
    } else if (warp != 3 && rank == 0) {
      // Two warps take every other block each: a block's waits, MMAs and commit take one of them longer to issue than the MMAs
      // of a narrow tile take to run.
      const ff::OperandForm form = ff::operand_form(true);
      const int own_tiles = tile0 < tiles ? (tiles - tile0 + tile_step - 1) / tile_step : 0;
      const int64_t all = static_cast<int64_t>(own_tiles) * blocks;
#pragma unroll 1
      for (int64_t use = warp - 1; use < all; use += 2) {
        const uint32_t b = static_cast<uint32_t>(use) % kBuffers, parity = (static_cast<uint32_t>(use) / kBuffers & 1u) ^ 1u;
        const uint32_t st = base + static_cast<uint32_t>(s) * kSlotBytes;
        const uint64_t da = ff::with_address(form, st), db = ff::with_address(form, st + kABytes);
        ok = __all_sync(0xffffffffu, wait_counted(full(s), phase, status) && wait_counted(acc_empty + 8u * b, parity, status));
        if (!ok) break;
        tc::tc_fence_after();
        mma_block<2>(tmem + b * kBn, da, db, p.idesc);
        if (ff::elect_one()) tc::mma_commit_pair(empty(s));
        __syncwarp();
        next(2);
      }
      // Every MMA issued above ends before TMEM is released.
      if (ff::elect_one()) tc::mma_commit<2>(mma_done);
      __syncwarp();
      wait_counted(mma_done, 0u, status);
    } else if (warp == 3) {
      // Scales of this CTA's rows, and of the tile's columns: of each (VECTOR) or of each group of 128.
      constexpr int kColumns = VECTOR ? kBn : (kBn + kBlock - 1) / kBlock;
      const int columns = VECTOR ? p.N : (p.N + kBlock - 1) / kBlock;
      uint32_t use = 0;
      for (int t = tile0; ok && t < tiles; t += tile_step) {
        int m0, n0;
        tc::tile_origin(t, p.tiles_m, p.tiles_n, 2 * kRows, kBn, m0, n0);
        m0 += rank * kRows;
        if (!VECTOR) n0 /= kBlock;
        const float* sa = p.sa.p + static_cast<int64_t>(m0) * p.sa.row;
        const float* sb = p.sb.p + static_cast<int64_t>(n0) * p.sb.row;
#pragma unroll 1
        for (int kb = 0; kb < blocks; kb += kScaleBlocks, ++use) {
          const uint32_t slot_of = use % kScaleSlots;
          ok = __all_sync(0xffffffffu, wait_counted(scale_empty + 8u * slot_of, ((use / kScaleSlots) & 1u) ^ 1u, status));
          if (!ok) break;
          uint32_t at = scales + slot_of * kScaleBytes;
#pragma unroll 1
          for (int j = kb; j < min(kb + kScaleBlocks, blocks); ++j, at += kBlockScales, sa += p.sa.block, sb += p.sb.block) {
            copy_scales<kRows>(at, sa, p.sa, p.sa_wide, m0, p.M, lane);
            copy_scales<kColumns>(at + 4u * kRows, sb, p.sb, VECTOR && p.sb_wide, n0, columns, lane);
          }
          cp_async_arrive_noinc(scale_full + 8u * slot_of);
        }
      }
      asm volatile("cp.async.wait_all;" ::: "memory");  // before the CTA may go
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSumRegs));
    const int e = warp - 4, q = warp & 3, half = e >> 2;  // quarter of the rows, half of the columns
    const uint32_t box = staging + static_cast<uint32_t>(e) * kStagingBytes;
    const uint32_t rows_at = tmem + (static_cast<uint32_t>(32 * q) << 16) + static_cast<uint32_t>(half * kWarpN);
    const uint32_t acc_empty_0 = tc::map_to_rank(acc_empty, 0);
    uint32_t use = 0, scale_use = 0, slot_at = 0, slot_phase = 0;
    bool ok = true;
    for (int t = tile0; ok && t < tiles; t += tile_step) {
      int m0, n0;
      tc::tile_origin(t, p.tiles_m, p.tiles_n, 2 * kRows, kBn, m0, n0);
      n0 += half * kWarpN;
      const int m = m0 + rank * kRows + 32 * q;
      uint64_t sum[CHUNKS][kChunk / 2];
#pragma unroll
      for (int u = 0; u < CHUNKS; ++u)
#pragma unroll
        for (int i = 0; i < kChunk / 2; ++i) sum[u][i] = 0;
#pragma unroll 1
      for (int kb = 0; ok && kb < blocks; kb += kScaleBlocks, ++scale_use) {
        const uint32_t ss = scale_use % kScaleSlots, from = scales + ss * kScaleBytes;
        ok = __all_sync(0xffffffffu, wait_counted(scale_full + 8u * ss, (scale_use / kScaleSlots) & 1u, status));
        if (!ok) break;
#pragma unroll 1
        for (int j = 0; j < kScaleBlocks && kb + j < blocks; ++j, ++use) {
          // This lane's row's scale, times that of the warp's columns where they share one (they lie within one group of 128).
          const uint32_t b = use % kBuffers, at = from + j * kBlockScales;
          const uint32_t columns = at + 4u * (kRows + (VECTOR ? half * kWarpN : half * kWarpN / kBlock));
          float a, g = 1.0f;
          asm volatile("ld.shared.f32 %0, [%1];" : "=f"(a) : "r"(at + 4u * (32 * q + lane)) : "memory");
          if (!VECTOR) asm volatile("ld.shared.f32 %0, [%1];" : "=f"(g) : "r"(columns) : "memory");
          ok = __all_sync(0xffffffffu, wait_counted(empty(0) + 8u * slot_at, slot_phase, status));
          if (++slot_at == kStages) {
            slot_at = 0;
            slot_phase ^= 1u;
          }
          if (!ok) break;
          tc::tc_fence_after();
          const uint32_t acc = rows_at + b * kBn;
          const uint64_t row = ff::both(VECTOR ? a : a * g);
#pragma unroll
          for (int u = 0; u < CHUNKS; ++u) {
            uint32_t x[kChunk];
            ff::load_columns(acc + u * kChunk, x);
            // The columns' scales come while the sums do.
            uint64_t w[VECTOR ? kChunk / 2 : 1];
            if constexpr (VECTOR) {
#pragma unroll
              for (int i = 0; i < kChunk / 2; i += 2) lds128_pairs(columns + 4u * (u * kChunk + 2 * i), w[i], w[i + 1]);
            }
            ff::wait_columns(x);
            if (u + 1 == CHUNKS) {
              tc::tc_fence_before();
              __syncwarp();
              if (lane == 0) ff::arrive_remote(acc_empty_0 + 8u * b);
            }
            uint64_t* to = sum[u];
            // Column, then row: scale by scale first, which would take any two scales whose product is normal, a 4096^3 product
            // takes 97 us instead of 87, and 103 to 121 with a second way that is taken for far scales only.
            if constexpr (VECTOR) {
#pragma unroll
              for (int i = 0; i < kChunk / 2; ++i)
                to[i] = ff::fma2(ff::mul2(pack2(__uint_as_float(x[2 * i]), __uint_as_float(x[2 * i + 1])), w[i]), row, to[i]);
            } else {
#pragma unroll
              for (int i = 0; i < kChunk / 2; ++i)
                to[i] = ff::fma2(pack2(__uint_as_float(x[2 * i]), __uint_as_float(x[2 * i + 1])), row, to[i]);
            }
          }
        }
        if (!ok) break;
        __syncwarp();
        if (lane == 0) mbar_arrive(scale_empty + 8u * ss);
      }
      if (!ok) break;
      constexpr int kColumns = box_columns<TYPE>();
#pragma unroll
      for (int c = 0; c < kWarpN; c += kColumns) {
        if (m >= p.M || n0 + c >= p.N) break;
        if (lane == 0) bulk_wait_read_all();
        __syncwarp();
        put_row<TYPE>(box, lane, sum[c / kChunk] + c % kChunk / 2);
        store_box<TYPE>(p, box, m, n0 + c, lane);
      }
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
template <int TYPE, int CHUNKS, bool VECTOR>
cudaError_t resident_clusters(int* out) {
  constexpr int kMaxDevices = 64;
  static std::atomic<int> known[kMaxDevices];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
  int n = known[dev].load(std::memory_order_acquire);
  if (n == 0) {
    auto kern = fp8_pair_kernel<TYPE, CHUNKS, VECTOR>;
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

template <int TYPE, int CHUNKS, bool VECTOR>
cudaError_t launch(const ProductTask& t, cudaStream_t stream, unsigned* status) {
  constexpr int kBn = 2 * CHUNKS * kChunk, kColumns = box_columns<TYPE>();
  constexpr int kBytes = TYPE == kF32 ? 4 : 2;
  int resident = 0;
  cudaError_t e = resident_clusters<TYPE, CHUNKS, VECTOR>(&resident);
  if (e != cudaSuccess) return e;
  PairParams p;
  memset(&p, 0, sizeof(p));
  p.sa = t.sa, p.sb = t.sb, p.sa_wide = wide_scales(t.sa), p.sb_wide = wide_scales(t.sb);
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
    e = TYPE == kF32 ? encode_tmap_f32_2d(&p.c, t.C, t.N, t.M, t.ldc, kColumns, 32, CU_TENSOR_MAP_SWIZZLE_64B)
                     : encode_tmap_16bit_2d(&p.c, t.C, t.N, t.M, t.ldc, kColumns, 32, CU_TENSOR_MAP_SWIZZLE_64B);
    if (e != cudaSuccess) return e;
  }
  const int64_t tiles = tiles_m * tiles_n;
  const ff::LaunchShape shape{dim3(static_cast<unsigned>(2 * (tiles < resident ? tiles : resident))), kThreads, 2, kSmemBytes};
  return ff::launch_early(stream, shape, fp8_pair_kernel<TYPE, CHUNKS, VECTOR>, p);
}

template <int TYPE, int CHUNKS>
cudaError_t launch_scales(const ProductTask& t, cudaStream_t stream, unsigned* status) {
  return t.b_group == 1 ? launch<TYPE, CHUNKS, true>(t, stream, status) : launch<TYPE, CHUNKS, false>(t, stream, status);
}

template <int TYPE>
cudaError_t launch_width(const ProductTask& t, int width, cudaStream_t stream, unsigned* status) {
  return width == 256 ? launch_scales<TYPE, 4>(t, stream, status)
                      : width == 128 ? launch_scales<TYPE, 2>(t, stream, status) : launch_scales<TYPE, 1>(t, stream, status);
}

}  // namespace

// The tile width with the shortest rounds of all pairs of SMs: a block of 128 of K takes a pair 0.21, 0.27 or 0.40 us in
// tiles of 64, 128 or 256 columns (with a scale for every column 0.28, 0.37, 0.62), a tile's end 0.3, 0.6 or 1.2 us, a
// launch 3.2. Measured in the three widths: 256 x 4096 x 4096 (N last) 10.5, 12.2 and 16.8 us, 512 x 4096 x 4096 17.1, 12.7
// and 16.9, 4096 x 4096 x 4096 99, 66 and 59.6.
PairPlan plan_pair(const ProductTask& t, int pairs) {
  static constexpr int kWidths[] = {256, 128, 64};
  static constexpr double kBlockTime[2][3] = {{0.40, 0.27, 0.21}, {0.62, 0.37, 0.28}};
  static constexpr double kTileTime[3] = {1.2, 0.6, 0.3};
  PairPlan best;
  for (int i = 0; i < 3; ++i) {
    const int64_t tiles = (t.M + 2 * kRows - 1) / (2 * kRows) * ((t.N + kWidths[i] - 1) / kWidths[i]);
    const double time = 3.2 + static_cast<double>((tiles + pairs - 1) / pairs) *
                                  (static_cast<double>(blocks_of(t.K)) * kBlockTime[t.b_group == 1][i] + kTileTime[i]);
    if (best.width == 0 || time < best.cost) {
      best.width = kWidths[i];
      best.cost = time;
    }
  }
  return best;
}

cudaError_t run_pair(const ProductTask& t, const PairPlan& plan, cudaStream_t stream, unsigned* status) {
  const int width = plan.width;
  return t.type == kF32 ? launch_width<kF32>(t, width, stream, status)
                        : t.type == kBf16 ? launch_width<kBf16>(t, width, stream, status)
                                          : launch_width<kF16>(t, width, stream, status);
}

}  // namespace fp8
}  // namespace t2s
