// fp8_rows.cu -- products of 8-bit operands with a scale for each block of 128 of K, where the outputs are too few to
// fill the SMs with the tiles of fp8_pair.cu: single tokens, small batches, small weights.
//
// The rows of B (a weight's outputs) lie along the tensor core's 128 rows and the rows of A along its columns (16, 32
// or 64 of them), so one token costs one pass over the weight and no more. The sum over K is split over the CTAs of a
// cluster (up to 8). Each takes its blocks' sums out of TMEM one after another (from four accumulators in turn),
// multiplies them by both scales and adds them in registers, then leaves its share in shared memory, and after a
// cluster barrier every CTA adds the shares of its part of the rows in rank order through distributed shared memory and
// stores. One launch, no workspace, the same bits every time.
//
// Measured: 1 x 4096 x 8192 (outputs last) 9.2 us, 3.7 TB/s of weights out of HBM, 64 x 4096 x 4096 8.4: about 4 us are the
// launch, the first blocks' latency and the join; 64 x 8192 x 28672 55, in two rounds of CTAs (224 tiles, one to an SM; its
// bytes take 35), 32 x 8192 x 28672 45. On SM pairs one row took 32 us, without a split of K 18.
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

constexpr int kTileN = 128;  // rows of B of a tile: the MMA's rows
constexpr int kWeightBytes = kTileN * kBlock;
constexpr int kThreads = 256;
constexpr int kSumWarps = 4;
constexpr int kMaxSplits = 8;
constexpr int kMaxStages = 12;
constexpr int kScaleBlocks = 4;  // blocks whose scales come to shared memory together
constexpr int kScaleSlots = 2;
constexpr int kBuffers = 4;  // accumulators

struct RowsParams {
  CUtensorMap w, x;
  Scales sa, sb;
  void* C;
  int64_t ldc;
  int M, N, blocks, tiles_n, stages, splits;
  int b_group, sa_wide, sb_wide;
  uint32_t idesc, stage_bytes;
  unsigned* status;
};

// TM: rows of A in a tile.
template <int TM>
struct Shape {
  static constexpr uint32_t kColumns = kBuffers * TM;  // of TMEM
  static constexpr int kStageBytes = kWeightBytes + TM * kBlock;
  static constexpr int kBlockScales = (kTileN + TM) * 4;  // of one block
  static constexpr int kScaleBytes = kScaleBlocks * kBlockScales;
  static constexpr int kShareBytes = TM * kTileN * 4;  // the sums that are joined lie over the ring
};

__device__ __forceinline__ float4 ld_cluster_v4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr));
  return v;
}

// Four neighbouring outputs of a row, `left` of them inside it.
template <int TYPE>
__device__ __forceinline__ void store4(void* c, int64_t at, int left, const float (&v)[4]) {
  if constexpr (TYPE == kF32) {
    float* p = static_cast<float*>(c) + at;
    if (left >= 4 && (reinterpret_cast<uintptr_t>(p) & 15u) == 0) {
      *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (i < left) p[i] = v[i];
    }
  } else {
    constexpr int kKind = TYPE == kBf16 ? ff::kBf16 : ff::kF16;
    uint16_t* p = static_cast<uint16_t*>(c) + at;
    if (left >= 4 && (reinterpret_cast<uintptr_t>(p) & 7u) == 0) {
      *reinterpret_cast<uint2*>(p) = make_uint2(ff::pack_f32<kKind>(v[0], v[1]), ff::pack_f32<kKind>(v[2], v[3]));
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (i < left) p[i] = ff::from_f32<kKind>(v[i]);
    }
  }
}

// Adds the S CTAs' shares and stores: the tile's rows in turn over the cluster's warps, four columns per lane, several
// rows' loads (distributed shared memory answers after hundreds of cycles) before the first sum.
template <int TYPE, int TM, int S>
__device__ __forceinline__ void finish(const RowsParams& p, uint32_t base, int rank, int n0, int m0) {
  constexpr int kUnroll = S <= 2 ? 4 : S == 4 ? 2 : 1;
  constexpr int kWarps = kThreads / 32, kStep = kWarps * S;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int n = n0 + 4 * lane, left = p.N - n, rows = min(TM, p.M - m0);
  uint32_t from[S];
#pragma unroll
  for (int i = 0; i < S; ++i) from[i] = S > 1 ? tc::map_to_rank(base + 16u * lane, i) : base + 16u * lane;
  for (int c0 = warp * S + rank; c0 < rows; c0 += kUnroll * kStep) {
    float4 parts[kUnroll][S];
#pragma unroll
    for (int j = 0; j < kUnroll; ++j) {
      const int c = min(c0 + j * kStep, rows - 1);
#pragma unroll
      for (int i = 0; i < S; ++i) {
        const uint32_t at = from[i] + static_cast<uint32_t>(c) * (kTileN * 4u);
        parts[j][i] = S > 1 ? ld_cluster_v4(at) : lds128(at);
      }
    }
#pragma unroll
    for (int j = 0; j < kUnroll; ++j) {
      const int c = c0 + j * kStep;
      if (c >= rows || left <= 0) break;
      float v[4] = {parts[j][0].x, parts[j][0].y, parts[j][0].z, parts[j][0].w};
#pragma unroll
      for (int i = 1; i < S; ++i)
        v[0] += parts[j][i].x, v[1] += parts[j][i].y, v[2] += parts[j][i].z, v[3] += parts[j][i].w;
      store4<TYPE>(p.C, (m0 + static_cast<int64_t>(c)) * p.ldc + n, left, v);
    }
  }
}

// Warp 0 copies the operands' blocks, warp 1 issues the MMAs, warp 2 copies scales, warps 4..7 take the sums; then
// all eight finish the outputs. full[s] / empty[s] per ring slot (empty also says that the slot's sums are in TMEM),
// acc_empty[b] per accumulator, scale_full[s] / scale_empty[s] per slot of scales. A role that gives up a bounded wait
// records it and stops; every thread still reaches the cluster barriers.
template <int TYPE, int TM>
__global__ void __launch_bounds__(kThreads) fp8_rows_kernel(const __grid_constant__ RowsParams p) {
  using T = Shape<TM>;
  extern __shared__ uint8_t smem_raw[];
  const int splits = p.splits, tile = static_cast<int>(blockIdx.x) / splits, stages = p.stages;
  const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
  const uint32_t ring_bytes = max(static_cast<uint32_t>(stages) * T::kStageBytes, static_cast<uint32_t>(T::kShareBytes));
  const uint32_t bars = base + ring_bytes;
  auto full = [&](int s) { return bars + 8u * s; };
  auto empty = [&](int s) { return bars + 8u * (kMaxStages + s); };
  const uint32_t acc_empty = bars + 16u * kMaxStages, scale_full = acc_empty + 8u * kBuffers;
  const uint32_t scale_empty = scale_full + 8u * kScaleSlots, done = scale_empty + 8u * kScaleSlots, slot = done + 8u;
  const uint32_t scales = bars + 512u;
  unsigned* const status = p.status;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = splits > 1 ? static_cast<int>(cluster_ctarank()) : 0;
  const int n0 = tile % p.tiles_n * kTileN, m0 = tile / p.tiles_n * TM;
  // This CTA's blocks of K.
  const int kb0 = static_cast<int>(static_cast<int64_t>(p.blocks) * rank / splits);
  const int kb1 = static_cast<int>(static_cast<int64_t>(p.blocks) * (rank + 1) / splits);

  if (threadIdx.x == 0) {
    for (int s = 0; s < stages; ++s) {
      mbar_init(full(s), 1);
      mbar_init(empty(s), 1);
    }
    for (int b = 0; b < kBuffers; ++b) mbar_init(acc_empty + 8u * b, kSumWarps);
    for (int s = 0; s < kScaleSlots; ++s) {
      mbar_init(scale_full + 8u * s, 32);
      mbar_init(scale_empty + 8u * s, kSumWarps);
    }
    mbar_init(done, 1);
    mbar_fence_init();
  }
  if (warp == 0 && ff::elect_one()) {
    tma_prefetch_desc(&p.w);
    tma_prefetch_desc(&p.x);
  }
  if (warp == 3) tc::tmem_alloc<1>(slot, T::kColumns);
  tc::tc_fence_before();
  __syncthreads();
  ff::wait_for_earlier_kernels();
  tc::tc_fence_after();
  uint32_t tmem;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(tmem) : "r"(slot) : "memory");

  int s = 0;
  uint32_t phase = 0;
  auto next = [&] {
    if (++s == stages) {
      s = 0;
      phase ^= 1u;
    }
  };
  bool ok = true;
  uint64_t sum[TM / 2];
#pragma unroll
  for (int i = 0; i < TM / 2; ++i) sum[i] = 0;
  if (warp == 0) {
#pragma unroll 1
    for (int kb = kb0; kb < kb1; ++kb) {
      ok = __all_sync(0xffffffffu, wait_counted(empty(s), phase ^ 1u, status));
      if (!ok) break;
      if (ff::elect_one()) {
        const uint32_t st = base + static_cast<uint32_t>(s) * T::kStageBytes;
        mbar_arrive_expect_tx(full(s), T::kStageBytes);
        tma_load_2d(st, &p.w, kb * kBlock, n0, full(s));
        tma_load_2d(st + kWeightBytes, &p.x, kb * kBlock, m0, full(s));
      }
      __syncwarp();
      next();
    }
  } else if (warp == 1) {
    const ff::OperandForm form = ff::operand_form(true);
    uint32_t use = 0;
#pragma unroll 1
    for (int kb = kb0; kb < kb1; ++kb, ++use) {
      const uint32_t b = use % kBuffers, st = base + static_cast<uint32_t>(s) * T::kStageBytes;
      const uint64_t dw = ff::with_address(form, st), dx = ff::with_address(form, st + kWeightBytes);
      ok = __all_sync(0xffffffffu, wait_counted(full(s), phase, status) &&
                                       wait_counted(acc_empty + 8u * b, (use / kBuffers & 1u) ^ 1u, status));
      if (!ok) break;
      tc::tc_fence_after();
      mma_block<1>(tmem + b * TM, dw, dx, p.idesc);
      if (ff::elect_one()) tc::mma_commit<1>(empty(s));
      __syncwarp();
      next();
    }
    if (ff::elect_one()) tc::mma_commit<1>(done);
    __syncwarp();
  } else if (warp == 2) {
    // Scales of the tile's rows of B (of each, or one for all 128) and of its rows of A.
    const bool each = p.b_group == 1;
    const int first = each ? n0 : n0 / kBlock;
    const float* sb = p.sb.p + first * p.sb.row + kb0 * p.sb.block;
    const float* sa = p.sa.p + m0 * p.sa.row + kb0 * p.sa.block;
    uint32_t use = 0;
#pragma unroll 1
    for (int kb = kb0; kb < kb1; kb += kScaleBlocks, ++use) {
      uint32_t at = scales + use % kScaleSlots * T::kScaleBytes;
      ok = __all_sync(0xffffffffu, wait_counted(scale_empty + 8u * (use % kScaleSlots), (use / kScaleSlots & 1u) ^ 1u, status));
      if (!ok) break;
#pragma unroll 1
      for (int j = kb; j < min(kb + kScaleBlocks, kb1); ++j, at += T::kBlockScales, sa += p.sa.block, sb += p.sb.block) {
        if (each) {
          copy_scales<kTileN>(at, sb, p.sb, p.sb_wide, first, p.N, lane);
        } else {
          copy_scales<1>(at, sb, p.sb, false, first, first + 1, lane);
        }
        copy_scales<TM>(at + 4u * kTileN, sa, p.sa, p.sa_wide, m0, p.M, lane);
      }
      cp_async_arrive_noinc(scale_full + 8u * (use % kScaleSlots));
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
  } else if (warp >= 4) {
    const int q = warp - 4;
    const uint32_t rows_at = tmem + (static_cast<uint32_t>(32 * q) << 16);
    uint32_t use = 0, scale_use = 0;
#pragma unroll 1
    for (int kb = kb0; ok && kb < kb1; kb += kScaleBlocks, ++scale_use) {
      const uint32_t ss = scale_use % kScaleSlots, at = scales + ss * T::kScaleBytes;
      ok = __all_sync(0xffffffffu, wait_counted(scale_full + 8u * ss, scale_use / kScaleSlots & 1u, status));
      if (!ok) break;
#pragma unroll 1
      for (int j = 0; j < kScaleBlocks && kb + j < kb1; ++j, ++use) {
        const uint32_t b = use % kBuffers, of_rows = at + j * T::kBlockScales, columns = of_rows + 4u * kTileN;
        float w;
        asm volatile("ld.shared.f32 %0, [%1];" : "=f"(w) : "r"(of_rows + (p.b_group == 1 ? 4u * (32 * q + lane) : 0u)) : "memory");
        ok = __all_sync(0xffffffffu, wait_counted(empty(s), phase, status));
        if (!ok) break;
        next();
        tc::tc_fence_after();
        const uint64_t row = ff::both(w);
#pragma unroll
        for (int c = 0; c < TM; c += 16) {
          uint32_t x[16];
          tc::tmem_ld16(rows_at + b * TM + c, x);
#pragma unroll
          for (int i = 0; i < 16; ++i) asm volatile("" : "+r"(x[i]));  // no use before the load's wait
          if (c + 16 == TM) {
            tc::tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(acc_empty + 8u * b);
          }
#pragma unroll
          for (int i = 0; i < 16; i += 4) {
            uint64_t lo, hi;
            lds128_pairs(columns + 4u * (c + i), lo, hi);
            uint64_t* to = sum + (c + i) / 2;
            to[0] = ff::fma2(ff::mul2(pack2(__uint_as_float(x[i]), __uint_as_float(x[i + 1])), lo), row, to[0]);
            to[1] = ff::fma2(ff::mul2(pack2(__uint_as_float(x[i + 2]), __uint_as_float(x[i + 3])), hi), row, to[1]);
          }
        }
      }
      if (!ok) break;
      __syncwarp();
      if (lane == 0) mbar_arrive(scale_empty + 8u * ss);
    }
  }

  // The shares, column by column (a row of A each), over the ring: all copies have been read by MMAs that are done.
  wait_counted(done, 0u, status);
  __syncthreads();
  if (warp >= 4) {
    const uint32_t to = base + 4u * (32 * (warp - 4) + lane);
#pragma unroll
    for (int c = 0; c < TM; c += 2) {
      const float2 v = ff::halves(sum[c / 2]);
      asm volatile("st.shared.f32 [%0], %1;" ::"r"(to + static_cast<uint32_t>(c) * (kTileN * 4u)), "f"(v.x) : "memory");
      asm volatile("st.shared.f32 [%0], %1;" ::"r"(to + static_cast<uint32_t>(c + 1) * (kTileN * 4u)), "f"(v.y) : "memory");
    }
  }
  tc::tc_fence_before();
  if (splits > 1) {
    cluster_sync_all();
  } else {
    __syncthreads();
  }
  switch (splits) {
    case 1: finish<TYPE, TM, 1>(p, base, rank, n0, m0); break;
    case 2: finish<TYPE, TM, 2>(p, base, rank, n0, m0); break;
    case 4: finish<TYPE, TM, 4>(p, base, rank, n0, m0); break;
    default: finish<TYPE, TM, 8>(p, base, rank, n0, m0); break;
  }
  // No CTA's shares go while another may read them.
  if (splits > 1) {
    cluster_sync_all();
  } else {
    __syncthreads();
  }
  if (warp == 3) {
    tc::tc_fence_after();
    tc::tmem_dealloc<1>(tmem, T::kColumns);
  }
}

template <int TYPE, int TM>
cudaError_t launch(const ProductTask& t, const RowsPlan& plan, cudaStream_t stream, unsigned* status) {
  using T = Shape<TM>;
  constexpr int kMaxDevices = 64;
  static std::atomic<bool> prepared[kMaxDevices];
  auto kern = fp8_rows_kernel<TYPE, TM>;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
  if (!prepared[dev].load(std::memory_order_acquire)) {
    if ((e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, 227 * 1024)) != cudaSuccess) return e;
    prepared[dev].store(true, std::memory_order_release);
  }
  RowsParams p;
  memset(&p, 0, sizeof(p));
  p.sa = t.sa, p.sb = t.sb, p.b_group = t.b_group, p.sa_wide = wide_scales(t.sa), p.sb_wide = wide_scales(t.sb);
  p.C = t.C, p.ldc = t.ldc;
  p.M = static_cast<int>(t.M), p.N = static_cast<int>(t.N);
  p.blocks = static_cast<int>(blocks_of(t.K));
  p.tiles_n = static_cast<int>((t.N + kTileN - 1) / kTileN);
  p.splits = plan.splits;
  p.idesc = instruction(t.format_b, t.format_a, kTileN, TM);
  p.status = status;
  const int64_t tiles = p.tiles_n * ((t.M + TM - 1) / TM);
  if (tiles * plan.splits > 0x7fffffff) return cudaErrorInvalidConfiguration;
  if (p.blocks > 0) {
    if ((e = encode_tmap_8bit_2d(&p.w, t.B, t.K, t.N, t.ldb, kBlock, kTileN, CU_TENSOR_MAP_SWIZZLE_128B)) != cudaSuccess)
      return e;
    if ((e = encode_tmap_8bit_2d(&p.x, t.A, t.K, t.M, t.lda, kBlock, TM, CU_TENSOR_MAP_SWIZZLE_128B)) != cudaSuccess) return e;
  }
  // Half of an SM's memory where more CTAs are to come or a ring of half is deep enough, otherwise all of it. (Tiles of 64 rows
  // do not come two to an SM all the same: the least share below is half of a CTA's limit, and the system takes 1 KB of each.)
  constexpr int kAround = 1024 + 512 + kScaleSlots * T::kScaleBytes;
  const int per_cta = (p.blocks + plan.splits - 1) / plan.splits;
  const int budget = (tiles * plan.splits > plan.reach || 6 * T::kStageBytes <= 112 * 1024 - kAround ? 112 : 216) * 1024 - kAround;
  int stages = budget / T::kStageBytes;
  if (stages > kMaxStages) stages = kMaxStages;
  if (stages > per_cta) stages = per_cta;
  if (stages < kBuffers) stages = kBuffers;  // empty[s] says for one block at a time that its sums are there
  p.stages = stages;
  int smem = stages * T::kStageBytes;
  if (smem < T::kShareBytes) smem = T::kShareBytes;
  smem += kAround;
  // CTAs that share an SM must find TMEM for all of them: shared memory in the proportion of TMEM, and never so little
  // that a CTA fits beside a kernel that fills the rest.
  const int share = static_cast<int>(227 * 1024 * static_cast<int64_t>(T::kColumns) / 512);
  if (smem < share) smem = share;
  if (smem < 48 * 1024) smem = 48 * 1024;
  return ff::launch_early(stream, {dim3(static_cast<unsigned>(tiles * plan.splits)), kThreads, plan.splits, smem}, kern, p);
}

template <int TYPE>
cudaError_t launch_rows(const ProductTask& t, const RowsPlan& plan, cudaStream_t stream, unsigned* status) {
  switch (plan.rows) {
    case 16: return launch<TYPE, 16>(t, plan, stream, status);
    case 32: return launch<TYPE, 32>(t, plan, stream, status);
    default: return launch<TYPE, 64>(t, plan, stream, status);
  }
}

}  // namespace

// Expected time in microseconds: what a launch takes, a CTA's blocks (0.27, 0.30 or 0.36 each in tiles of 16, 32 or 64
// rows, measured) and the join, in as many waves as the CTAs need; all SMs together take in at most 14 TB/s. Against the
// pairs' kernel: 64 x 4096 x 4096 8.4 us here and 10.3 there, 128 x 4096 x 4096 10.3 and 10.4, 256 x 4096 x 4096 14.5 and
// 10.5.
RowsPlan plan_rows(const ProductTask& t, int sms) {
  RowsPlan best;
  const int64_t blocks = blocks_of(t.K), tiles_n = (t.N + kTileN - 1) / kTileN;
  for (const int rows : {16, 32, 64}) {
    const int64_t tiles = tiles_n * ((t.M + rows - 1) / rows);
    const double block = rows == 16 ? 0.27 : rows == 32 ? 0.30 : 0.36;
    for (int splits = 1; splits <= kMaxSplits; splits *= 2) {
      if (splits > 1 && blocks < 2 * splits) break;
      // SMs that clusters reach when a CTA fills an SM.
      const int reach = splits <= 2 ? sms : splits == 4 ? sms * 95 / 100 : sms * 79 / 100;
      const double per_cta = static_cast<double>((blocks + splits - 1) / splits) * block + rows * 0.017;
      double time = per_cta + static_cast<double>((tiles * splits - 1) / reach) * (per_cta + 1.0);
      const double feed = static_cast<double>(tiles) * static_cast<double>(blocks) * (kWeightBytes + rows * kBlock) / 14e6;
      if (time < feed) time = feed;
      time += 4.0 + (splits > 1 ? 0.6 : 0.0);
      if (best.rows == 0 || time < best.cost) {
        best.rows = rows;
        best.splits = splits;
        best.reach = reach;
        best.cost = time;
      }
    }
    if (rows >= t.M) break;
  }
  return best;
}

cudaError_t run_rows(const ProductTask& t, const RowsPlan& plan, cudaStream_t stream, unsigned* status) {
  return t.type == kF32 ? launch_rows<kF32>(t, plan, stream, status)
                        : t.type == kBf16 ? launch_rows<kBf16>(t, plan, stream, status)
                                          : launch_rows<kF16>(t, plan, stream, status);
}

}  // namespace fp8
}  // namespace t2s
