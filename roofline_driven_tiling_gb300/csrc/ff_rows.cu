// ff_rows.cu -- the products of the feed-forward operators where the outputs are too few to fill the
// SMs with the tiles of ff_pair.cu: a few rows of X (single tokens, small batches), small weights.
//
// The weight's outputs lie along the tensor core's 128 rows and the rows of X along its columns
// (16 to 256 of them), so one token costs one pass over the weight and no more. The sum over K is
// split over the CTAs of a cluster (up to 8): each accumulates its K blocks in TMEM, leaves the
// partial sums in its shared memory, and after a cluster barrier every CTA adds the partial sums of
// its share of the rows, in rank order through distributed shared memory, applies the epilogue and
// stores. One launch, no workspace, the same bits every time.
#include <cuda.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>
#include <cstring>

#include "ff_device.cuh"
#include "ff_internal.h"
#include "ff_math.cuh"
#include "t2s_device.cuh"
#include "t2s_tmap.h"
#include "tc_gemm.cuh"

namespace t2s {
namespace ff {
namespace {

constexpr int kTileN = 128;  // outputs of a tile: the MMA's rows
constexpr int kWeightBytes = kTileN * kBK * 2;
constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
constexpr int kMaxSplits = 8;
constexpr int kMaxStages = 12;

struct RowsParams {
  CUtensorMap w[2], x[2];
  const uint16_t* bias;
  const uint16_t* R;
  uint16_t *Y, *Z, *Z2;
  int64_t ldr, ldy, ldz, ldz2;
  unsigned* status;
  int M, N;
  int nkb, nkb_first;  // K blocks, and how many of them come from w[0], x[0]
  int tm;              // rows of X in a tile: the MMA's N
  int splits, stages;
  int w_k_major, x_k_major, x_boxes;
  int act;
  uint32_t idesc, stage_bytes, tmem_cols;
};

__device__ __forceinline__ float4 ld_cluster_v4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr));
  return v;
}

// Four consecutive values of a row, zeros beyond its end.
template <int KIND>
__device__ __forceinline__ void load4(const uint16_t* p, int left, float (&v)[4]) {
  if (left >= 4 && (reinterpret_cast<uintptr_t>(p) & 7u) == 0) {
    const uint2 w = *reinterpret_cast<const uint2*>(p);
    const float2 a = to_f32x2<KIND>(w.x), b = to_f32x2<KIND>(w.y);
    v[0] = a.x, v[1] = a.y, v[2] = b.x, v[3] = b.y;
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = i < left ? to_f32<KIND>(p[i]) : 0.0f;
  }
}

template <int KIND>
__device__ __forceinline__ void store4(uint16_t* p, int left, const float (&v)[4]) {
  if (left >= 4 && (reinterpret_cast<uintptr_t>(p) & 7u) == 0) {
    *reinterpret_cast<uint2*>(p) = make_uint2(pack_f32<KIND>(v[0], v[1]), pack_f32<KIND>(v[2], v[3]));
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i < left) p[i] = from_f32<KIND>(v[i]);
  }
}

// Warp 0 copies the weight's blocks, warp 2 those of X (and of the gated form's second weight),
// warp 1 issues the MMAs; then all eight warps read TMEM and finish the outputs. full[s] / empty[s]
// per ring slot. A role that gives up a bounded wait records it and stops; every thread still
// reaches the cluster barriers.
template <int KIND, bool GATED>
__global__ void __launch_bounds__(kThreads) ff_rows_kernel(const __grid_constant__ RowsParams p) {
  extern __shared__ uint8_t smem_raw[];
  const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
  const int S = p.stages;
  const uint32_t bars = base + S * p.stage_bytes;
  auto full = [&](int s) { return bars + 8u * s; };
  auto empty = [&](int s) { return bars + 8u * (kMaxStages + s); };
  const uint32_t done = bars + 16u * kMaxStages, slot = done + 8u;
  unsigned* const status = p.status;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = p.splits > 1 ? static_cast<int>(cluster_ctarank()) : 0;
  const int n0 = static_cast<int>(blockIdx.x / p.splits) * kTileN, m0 = static_cast<int>(blockIdx.y) * p.tm;
  // This CTA's K blocks.
  const int kb0 = static_cast<int>(static_cast<int64_t>(p.nkb) * rank / p.splits);
  const int kb1 = static_cast<int>(static_cast<int64_t>(p.nkb) * (rank + 1) / p.splits);

  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(full(s), 1);
      mbar_init(empty(s), 1);
    }
    mbar_init(done, 1);
    mbar_fence_init();
  }
  if (warp == 3) tc::tmem_alloc<1>(slot, p.tmem_cols);
  tc::tc_fence_before();
  __syncthreads();
  wait_for_earlier_kernels();
  tc::tc_fence_after();
  uint32_t tmem;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(tmem) : "r"(slot) : "memory");
  constexpr int kWeights = GATED ? 2 : 1;
  constexpr uint32_t kXOffset = kWeights * kWeightBytes;

  if (warp == 0 || warp == 2) {
    {
      const bool is_w = warp == 0, k_major = p.w_k_major, x_k_major = p.x_k_major;
      const int first = p.nkb_first, x_boxes = p.x_boxes;
      const uint32_t expect = is_w ? p.stage_bytes : 0u;
      Ring ring(base + (is_w ? 0 : GATED ? kWeightBytes : kXOffset), p.stage_bytes, full(0), empty(0), S);
      // Joined products: K blocks before `first` from the first pair of operands, then the second.
      for (int part = 0; part < 2; ++part) {
        const int from = part ? max(kb0 - first, 0) : min(kb0, first), to = part ? kb1 - first : min(kb1, first);
        const CUtensorMap *mw = &p.w[GATED ? (is_w ? 0 : 1) : part], *mx = &p.x[part];
        if (from >= to) continue;
        bool ok;
        if (is_w && k_major) {
          ok = ring.copy(from, to, expect, full(0), status,
                         [&](uint32_t st, int k0, uint32_t bar) { tma_load_2d(st, mw, k0, n0, bar); });
        } else if (is_w) {
          ok = ring.copy(from, to, expect, full(0), status, [&](uint32_t st, int k0, uint32_t bar) {
            tma_load_2d(st, mw, n0, k0, bar);
            tma_load_2d(st + kBoxBytes, mw, n0 + 64, k0, bar);
          });
        } else {
          ok = ring.copy(from, to, expect, full(0), status, [&](uint32_t st, int k0, uint32_t bar) {
            if (GATED) {
              if (k_major) {
                tma_load_2d(st, mw, k0, n0, bar);
              } else {
                tma_load_2d(st, mw, n0, k0, bar);
                tma_load_2d(st + kBoxBytes, mw, n0 + 64, k0, bar);
              }
              st += kWeightBytes;
            }
            if (x_k_major) {
              tma_load_2d(st, mx, k0, m0, bar);
            } else {
              for (int j = 0; j < x_boxes; ++j) tma_load_2d(st + j * kBoxBytes, mx, m0 + 64 * j, k0, bar);
            }
          });
        }
        if (!ok) break;
      }
    }
  } else if (warp == 1) {
    {
      int s = 0;
      uint32_t phase = 0, st = base;
      const OperandForm fw = operand_form(p.w_k_major), fx = operand_form(p.x_k_major);
#pragma unroll 1
      for (int kb = kb0; kb < kb1; ++kb) {
        if (!__all_sync(0xffffffffu, wait_bounded(full(s), phase, status))) break;
        tc::tc_fence_after();
        const uint64_t dw = with_address(fw, st), dx = with_address(fx, st + kXOffset);
        mma_block<1>(tmem, dw, fw.step, dx, fx.step, p.idesc, kb - kb0);
        if (GATED) mma_block<1>(tmem + p.tm, dw + (kWeightBytes >> 4), fw.step, dx, fx.step, p.idesc, kb - kb0);
        if (elect_one()) tc::mma_commit<1>(empty(s));
        __syncwarp();
        st += p.stage_bytes;
        if (++s == S) {
          s = 0;
          st = base;
          phase ^= 1u;
        }
      }
      if (elect_one()) tc::mma_commit<1>(done);
    }
    __syncwarp();
  }

  // The partial sums, column by column (a row of X each), over the ring: all copies have been
  // read by MMAs that are done.
  wait_bounded(done, 0u, status);
  __syncwarp();
  tc::tc_fence_after();
  const bool any = kb1 > kb0;
  const uint32_t row = static_cast<uint32_t>(32 * (warp & 3));
  const int columns = kWeights * p.tm;  // gated: G's, then U's
  for (int c = (warp >> 2) * 16; c < columns; c += 32) {
    uint32_t r[16];
    tc::tmem_ld16(tmem + (row << 16) + static_cast<uint32_t>(c), r);
#pragma unroll
    for (int i = 0; i < 16; ++i)
      asm volatile("st.shared.b32 [%0], %1;" ::"r"(base + static_cast<uint32_t>(c + i) * (kTileN * 4u) +
                                                   (row + lane) * 4u),
                   "r"(any ? r[i] : 0u)
                   : "memory");
  }
  tc::tc_fence_before();
  if (p.splits > 1) {
    cluster_sync_all();
  } else {
    __syncthreads();
  }

  // Rows of X in turn over the cluster's warps; four outputs per lane.
  const int n = n0 + 4 * lane, left = p.N - n;
  const int rows = min(p.tm, p.M - m0);
  float bias[4] = {};
  if (p.bias != nullptr && left > 0) load4<KIND>(p.bias + n, left, bias);
  for (int c = warp * p.splits + rank; c < rows; c += kWarps * p.splits) {
    const int64_t m = m0 + c;
    float r[4] = {}, v[4] = {}, u[4] = {};
    if (p.R != nullptr && left > 0) load4<KIND>(p.R + m * p.ldr + n, left, r);
    const uint32_t at = base + static_cast<uint32_t>(c) * (kTileN * 4u) + 16u * lane;
    const uint32_t at_u = at + static_cast<uint32_t>(p.tm) * (kTileN * 4u);
    if (p.splits > 1) {
      float4 parts[kMaxSplits], parts_u[GATED ? kMaxSplits : 1];
#pragma unroll
      for (int i = 0; i < kMaxSplits; ++i)
        if (i < p.splits) {
          parts[i] = ld_cluster_v4(tc::map_to_rank(at, i));
          if (GATED) parts_u[i] = ld_cluster_v4(tc::map_to_rank(at_u, i));
        }
#pragma unroll
      for (int i = 0; i < kMaxSplits; ++i)
        if (i < p.splits) {
          v[0] += parts[i].x, v[1] += parts[i].y, v[2] += parts[i].z, v[3] += parts[i].w;
          if (GATED) u[0] += parts_u[i].x, u[1] += parts_u[i].y, u[2] += parts_u[i].z, u[3] += parts_u[i].w;
        }
    } else {
      const float4 a = lds128(at);
      v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
      if (GATED) {
        const float4 b = lds128(at_u);
        u[0] = b.x, u[1] = b.y, u[2] = b.z, u[3] = b.w;
      }
    }
    if (left <= 0) continue;
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] += bias[i];
    if (p.Z != nullptr) store4<KIND>(p.Z + m * p.ldz + n, left, v);
    if (GATED && p.Z2 != nullptr) store4<KIND>(p.Z2 + m * p.ldz2 + n, left, u);
    with_act(p.act, [&](auto a) {
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = act_value<decltype(a)::value>(v[i]);
    });
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = GATED ? v[i] * u[i] : v[i] + r[i];
    store4<KIND>(p.Y + m * p.ldy + n, left, v);
  }

  // No CTA's partial sums go while another may read them.
  if (p.splits > 1) {
    cluster_sync_all();
  } else {
    __syncthreads();
  }
  if (warp == 3) {
    tc::tc_fence_after();
    tc::tmem_dealloc<1>(tmem, p.tmem_cols);
  }
}

template <int KIND, bool GATED>
cudaError_t launch(const Context& c, const Task& t, const RowsPlan& plan) {
  constexpr int kMaxDevices = 64;
  constexpr int kMaxSmem = 227 * 1024;
  static std::atomic<bool> prepared[kMaxDevices];
  auto kern = ff_rows_kernel<KIND, GATED>;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
  if (!prepared[dev].load(std::memory_order_acquire)) {
    if ((e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxSmem)) != cudaSuccess)
      return e;
    prepared[dev].store(true, std::memory_order_release);
  }
  RowsParams p;
  memset(&p, 0, sizeof(p));
  p.status = c.status;
  p.M = static_cast<int>(t.M);
  p.N = static_cast<int>(t.N);
  p.tm = plan.tm;
  p.splits = plan.splits;
  p.stages = plan.stages;
  p.stage_bytes = plan.stage_bytes;
  p.tmem_cols = plan.tmem_cols;
  const int blocks = static_cast<int>((t.K + kBK - 1) / kBK);
  p.nkb_first = blocks;
  p.nkb = t.form == kJoined ? 2 * blocks : blocks;
  p.w_k_major = t.B.k_major;
  p.x_k_major = t.A.k_major;
  p.x_boxes = (plan.tm + 63) / 64;
  const uint32_t fmt = KIND == kBf16 ? 1u : 0u;
  // D FP32, both operands of the 16-bit type, their orders, N = tm, M = 128.
  p.idesc = (1u << 4) | (fmt << 7) | (fmt << 10) | ((p.w_k_major ? 0u : 1u) << 15) |
            ((p.x_k_major ? 0u : 1u) << 16) | (static_cast<uint32_t>(plan.tm >> 3) << 17) |
            (static_cast<uint32_t>(kTileN >> 4) << 24);
  p.bias = t.bias;
  p.R = t.R.p, p.ldr = t.R.ld;
  p.Y = t.Y.p, p.ldy = t.Y.ld;
  p.Z = t.Z.p, p.ldz = t.Z.ld;
  p.Z2 = t.Z2.p, p.ldz2 = t.Z2.ld;
  p.act = t.act;
  if (blocks > 0) {
    const uint32_t tm = static_cast<uint32_t>(plan.tm);
    if ((e = operand_map(&p.w[0], t.B, t.N, t.K, kTileN)) != cudaSuccess) return e;
    if ((e = operand_map(&p.x[0], t.A, t.M, t.K, tm)) != cudaSuccess) return e;
    if (t.form != kLinear && (e = operand_map(&p.w[1], t.B2, t.N, t.K, kTileN)) != cudaSuccess) return e;
    if (t.form == kJoined && (e = operand_map(&p.x[1], t.A2, t.M, t.K, tm)) != cudaSuccess) return e;
  }
  const LaunchShape shape{dim3(static_cast<unsigned>((t.N + kTileN - 1) / kTileN) * plan.splits,
                               static_cast<unsigned>((t.M + plan.tm - 1) / plan.tm)),
                          kThreads, plan.splits, plan.smem_bytes};
  return launch_early(c.stream, shape, kern, p);
}

}  // namespace

RowsPlan plan_rows(const Task& t, int sms) {
  RowsPlan plan;
  const int weights = t.form == kGated ? 2 : 1;
  // Rows of X per tile: equal shares of M, at most 256 sums per TMEM lane.
  const int64_t most = 256 / weights;
  const int64_t tiles_m = (t.M + most - 1) / most;
  plan.tm = static_cast<int>(((t.M + tiles_m - 1) / tiles_m + 15) / 16 * 16);
  const int64_t tiles = ((t.N + kTileN - 1) / kTileN) * ((t.M + plan.tm - 1) / plan.tm);
  const int64_t blocks = (t.K + kBK - 1) / kBK * (t.form == kJoined ? 2 : 1);
  // As many splits of K as leave two blocks to each CTA and one CTA to an SM. Of the SMs, clusters of
  // 4 reach 95 % and clusters of 8 79 % with CTAs that fill them (144 and 120 of 152).
  plan.splits = 1;
  for (int s = 2; s <= kMaxSplits; s *= 2) {
    const int64_t reach = s <= 2 ? sms : s == 4 ? sms * 95 / 100 : sms * 79 / 100;
    if (tiles * s <= reach && blocks >= 2 * s) plan.splits = s;
  }
  const int64_t ctas = tiles * plan.splits;
  plan.ctas = ctas;
  const int x_bytes = t.A.k_major ? plan.tm * kBK * 2 : (plan.tm + 63) / 64 * kBoxBytes;
  plan.stage_bytes = static_cast<uint32_t>(weights * kWeightBytes + x_bytes);
  plan.tmem_cols = 32;
  while (plan.tmem_cols < static_cast<uint32_t>(weights * plan.tm)) plan.tmem_cols *= 2;
  // One CTA per SM takes a deep ring, two share the SM's memory. The partial sums lie over the
  // ring, so it holds at least those.
  const int partials = weights * plan.tm * kTileN * 4;
  const int budget = (ctas > sms ? 112 : 200) * 1024;
  const int64_t per_cta = (blocks + plan.splits - 1) / plan.splits;
  int stages = static_cast<int>(budget / plan.stage_bytes);
  if (stages > kMaxStages) stages = kMaxStages;
  if (stages > per_cta) stages = static_cast<int>(per_cta);
  const int least = (partials + static_cast<int>(plan.stage_bytes) - 1) / static_cast<int>(plan.stage_bytes);
  if (stages < least) stages = least;
  plan.stages = stages;
  plan.smem_bytes = stages * static_cast<int>(plan.stage_bytes) + 1024 + 512;
  // CTAs that share an SM must find TMEM for all of them, or clusters could wait for each other's:
  // shared memory in the proportion of TMEM (and never so little that a CTA fits beside a kernel
  // that fills the rest) keeps the sum of their columns at most 512.
  const int share = static_cast<int>(227 * 1024 * static_cast<int64_t>(plan.tmem_cols) / 512);
  if (plan.smem_bytes < share) plan.smem_bytes = share;
  if (plan.smem_bytes < 48 * 1024) plan.smem_bytes = 48 * 1024;
  return plan;
}

cudaError_t run_rows(const Context& c, const Task& t, const RowsPlan& plan) {
  const bool gated = t.form == kGated;
  if (c.kind == kBf16) return gated ? launch<kBf16, true>(c, t, plan) : launch<kBf16, false>(c, t, plan);
  return gated ? launch<kF16, true>(c, t, plan) : launch<kF16, false>(c, t, plan);
}

}  // namespace ff
}  // namespace t2s
