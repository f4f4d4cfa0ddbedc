// ff_rows.cu -- the products of the feed-forward operators where the outputs are too few to fill the
// SMs with the tiles of ff_pair.cu: a few rows of X (single tokens, small batches), small weights.
//
// The weight's outputs lie along the tensor core's 128 rows and the rows of X along its columns
// (16 to 256 of them), so one token costs one pass over the weight and no more. The sum over K is
// split over the CTAs of a cluster (up to 8): each accumulates its K blocks in TMEM, leaves the
// partial sums in its shared memory, and after a cluster barrier every CTA adds the partial sums of
// its share of the rows, in rank order through distributed shared memory, applies the epilogue and
// stores. One launch (for up to three products of a gradient), no workspace, the same bits every
// time.
//
// What bounds it: one pass over the weight through HBM and what a launch takes around it, about 4 us
// (start-up, the ring's first block, two cluster barriers, the join). Rows x inputs x outputs on the device,
// weights from HBM (and, second, from the L2 cache, as a benchmark finds them that repeats one call):
// 1x4096x4096 8.4 us, 4.0 TB/s (6.2), 8x8192x4096 13.2, 5.1 TB/s (9.0), gated 1x4096x8192 22.3, 6.0 of the
// 6.7 TB/s that a copy reaches (larger than the L2), 64x4096x4096 10.3 (7.9), 256x4096x4096 15.2 (13.0). Without
// the split over K, on 32 SMs, 1x4096x4096 takes 14 from the L2 cache.
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

struct RowsProblem {
  CUtensorMap w[2], x[2];
  const uint16_t* bias;
  const uint16_t* R;
  uint16_t *Y, *Z, *Z2;
  int64_t ldr, ldy, ldz, ldz2;
  int M, N;
  int nkb, nkb_first;  // K blocks, and how many of them come from w[0], x[0]
  int tm;              // rows of X in a tile: the MMA's N
  int tiles_n, stages;
  int w_k_major, x_k_major, x_boxes;
  int act;
  uint32_t idesc, stage_bytes, tmem_cols;
};

struct RowsParams {
  RowsProblem p[kMaxProblems];
  int first[kMaxProblems];  // first tile of each problem (one past the last tile where there is none)
  int splits;
  unsigned* status;
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

// Adds the S CTAs' partial sums, applies the epilogue and stores: the rows of X in turn over the
// cluster's warps, four outputs per lane, several rows' loads (distributed shared memory and the
// residual answer after hundreds of cycles) before the first row's arithmetic.
template <int KIND, bool GATED, int S>
__device__ __forceinline__ void finish(const RowsProblem& p, uint32_t base, int rank, int n0, int m0) {
  constexpr int kWeights = GATED ? 2 : 1;
  constexpr int kUnroll = S * kWeights <= 2 ? 4 : S * kWeights <= 4 ? 2 : 1;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int n = n0 + 4 * lane, left = p.N - n, rows = min(p.tm, p.M - m0);
  float bias[4] = {};
  if (p.bias != nullptr && left > 0) load4<KIND>(p.bias + n, left, bias);
  uint32_t from[S];
#pragma unroll
  for (int i = 0; i < S; ++i) from[i] = S > 1 ? tc::map_to_rank(base + 16u * lane, i) : base + 16u * lane;
  constexpr int kStep = kWarps * S;
  for (int c0 = warp * S + rank; c0 < rows; c0 += kUnroll * kStep) {
    float4 parts[kUnroll][kWeights][S];
    float r[kUnroll][4] = {};
#pragma unroll
    for (int j = 0; j < kUnroll; ++j) {
      const int c = min(c0 + j * kStep, rows - 1);
      if (p.R != nullptr && left > 0) load4<KIND>(p.R + (m0 + static_cast<int64_t>(c)) * p.ldr + n, left, r[j]);
#pragma unroll
      for (int g = 0; g < kWeights; ++g)
#pragma unroll
        for (int i = 0; i < S; ++i) {
          const uint32_t at = from[i] + static_cast<uint32_t>(g * p.tm + c) * (kTileN * 4u);
          parts[j][g][i] = S > 1 ? ld_cluster_v4(at) : lds128(at);
        }
    }
    float v[kUnroll][kWeights][4], y[kUnroll][4];
#pragma unroll
    for (int j = 0; j < kUnroll; ++j)
#pragma unroll
      for (int g = 0; g < kWeights; ++g) {
        float* x = v[j][g];
        x[0] = parts[j][g][0].x, x[1] = parts[j][g][0].y, x[2] = parts[j][g][0].z, x[3] = parts[j][g][0].w;
#pragma unroll
        for (int i = 1; i < S; ++i)
          x[0] += parts[j][g][i].x, x[1] += parts[j][g][i].y, x[2] += parts[j][g][i].z, x[3] += parts[j][g][i].w;
        if (g == 0) x[0] += bias[0], x[1] += bias[1], x[2] += bias[2], x[3] += bias[3];
      }
    with_act(p.act, [&](auto a) {
#pragma unroll
      for (int j = 0; j < kUnroll; ++j)
#pragma unroll
        for (int i = 0; i < 4; i += 2) {
          const float2 x = halves(act_pair<decltype(a)::value>(pack2(v[j][0][i], v[j][0][i + 1])));
          y[j][i] = GATED ? x.x * v[j][kWeights - 1][i] : x.x + r[j][i];
          y[j][i + 1] = GATED ? x.y * v[j][kWeights - 1][i + 1] : x.y + r[j][i + 1];
        }
    });
    if (left <= 0) continue;
#pragma unroll
    for (int j = 0; j < kUnroll; ++j) {
      const int c = c0 + j * kStep;
      if (c >= rows) break;
      const int64_t m = m0 + static_cast<int64_t>(c);
      if (p.Z != nullptr) store4<KIND>(p.Z + m * p.ldz + n, left, v[j][0]);
      if (GATED && p.Z2 != nullptr) store4<KIND>(p.Z2 + m * p.ldz2 + n, left, v[j][kWeights - 1]);
      store4<KIND>(p.Y + m * p.ldy + n, left, y[j]);
    }
  }
}

// Warp 0 copies the weight's blocks, warp 2 those of X (and of the gated form's second weight),
// warp 1 issues the MMAs; then all eight warps read TMEM and finish the outputs. full[s] / empty[s]
// per ring slot. A role that gives up a bounded wait records it and stops; every thread still
// reaches the cluster barriers.
template <int KIND, bool GATED>
__global__ void __launch_bounds__(kThreads) ff_rows_kernel(const __grid_constant__ RowsParams params) {
  extern __shared__ uint8_t smem_raw[];
  const int splits = params.splits, cluster = static_cast<int>(blockIdx.x) / splits;
  const int pi = cluster < params.first[1] ? 0 : cluster < params.first[2] ? 1 : 2;
  const RowsProblem& p = params.p[pi];
  const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
  const int S = p.stages;
  const uint32_t bars = base + S * p.stage_bytes;
  auto full = [&](int s) { return bars + 8u * s; };
  auto empty = [&](int s) { return bars + 8u * (kMaxStages + s); };
  const uint32_t done = bars + 16u * kMaxStages, slot = done + 8u;
  unsigned* const status = params.status;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = splits > 1 ? static_cast<int>(cluster_ctarank()) : 0;
  const int tile = cluster - params.first[pi];
  const int n0 = tile % p.tiles_n * kTileN, m0 = tile / p.tiles_n * p.tm;
  // This CTA's K blocks.
  const int kb0 = static_cast<int>(static_cast<int64_t>(p.nkb) * rank / splits);
  const int kb1 = static_cast<int>(static_cast<int64_t>(p.nkb) * (rank + 1) / splits);

  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(full(s), 1);
      mbar_init(empty(s), 1);
    }
    mbar_init(done, 1);
    mbar_fence_init();
  }
  if (warp == 0 && elect_one()) tma_prefetch_desc(&p.w[0]);
  if (warp == 2 && elect_one()) tma_prefetch_desc(&p.x[0]);
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
      Ring ring(base + (is_w ? 0 : GATED ? kWeightBytes : kXOffset), p.stage_bytes, full(0), empty(0), S, kBK);
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
  if (splits > 1) {
    cluster_sync_all();
  } else {
    __syncthreads();
  }

  switch (splits) {
    case 1: finish<KIND, GATED, 1>(p, base, rank, n0, m0); break;
    case 2: finish<KIND, GATED, 2>(p, base, rank, n0, m0); break;
    case 4: finish<KIND, GATED, 4>(p, base, rank, n0, m0); break;
    default: finish<KIND, GATED, 8>(p, base, rank, n0, m0); break;
  }

  // No CTA's partial sums go while another may read them.
  if (splits > 1) {
    cluster_sync_all();
  } else {
    __syncthreads();
  }
  if (warp == 3) {
    tc::tc_fence_after();
    tc::tmem_dealloc<1>(tmem, p.tmem_cols);
  }
}

template <int KIND>
cudaError_t fill(RowsProblem* p, const Task& t, const RowsTile& tile) {
  cudaError_t e = cudaSuccess;
  p->M = static_cast<int>(t.M);
  p->N = static_cast<int>(t.N);
  p->tm = tile.tm;
  p->tiles_n = static_cast<int>((t.N + kTileN - 1) / kTileN);
  p->stages = tile.stages;
  p->stage_bytes = tile.stage_bytes;
  p->tmem_cols = tile.tmem_cols;
  const int blocks = static_cast<int>((t.K + kBK - 1) / kBK);
  p->nkb_first = blocks;
  p->nkb = t.form == kJoined ? 2 * blocks : blocks;
  p->w_k_major = t.B.k_major;
  p->x_k_major = t.A.k_major;
  p->x_boxes = (tile.tm + 63) / 64;
  const uint32_t fmt = KIND == kBf16 ? 1u : 0u;
  // D FP32, both operands of the 16-bit type, their orders, N = tm, M = 128.
  p->idesc = (1u << 4) | (fmt << 7) | (fmt << 10) | ((p->w_k_major ? 0u : 1u) << 15) |
             ((p->x_k_major ? 0u : 1u) << 16) | (static_cast<uint32_t>(tile.tm >> 3) << 17) |
             (static_cast<uint32_t>(kTileN >> 4) << 24);
  p->bias = t.bias;
  p->R = t.R.p, p->ldr = t.R.ld;
  p->Y = t.Y.p, p->ldy = t.Y.ld;
  p->Z = t.Z.p, p->ldz = t.Z.ld;
  p->Z2 = t.Z2.p, p->ldz2 = t.Z2.ld;
  p->act = t.act;
  if (blocks == 0) return cudaSuccess;
  const uint32_t tm = static_cast<uint32_t>(tile.tm);
  if ((e = operand_map(&p->w[0], t.B, t.N, t.K, kTileN)) != cudaSuccess) return e;
  if ((e = operand_map(&p->x[0], t.A, t.M, t.K, tm)) != cudaSuccess) return e;
  if (t.form != kLinear && (e = operand_map(&p->w[1], t.B2, t.N, t.K, kTileN)) != cudaSuccess) return e;
  if (t.form == kJoined && (e = operand_map(&p->x[1], t.A2, t.M, t.K, tm)) != cudaSuccess) return e;
  return cudaSuccess;
}

template <int KIND, bool GATED>
cudaError_t launch(const Context& c, const Task* tasks, const RowsPlan& plan, int n) {
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
  RowsParams params;
  memset(&params, 0, sizeof(params));
  params.status = c.status;
  params.splits = plan.splits;
  int64_t tiles = 0;
  for (int i = 0; i < kMaxProblems; ++i) {
    params.first[i] = static_cast<int>(tiles);
    if (i >= n) continue;
    if ((e = fill<KIND>(&params.p[i], tasks[i], plan.tile[i])) != cudaSuccess) return e;
    tiles += static_cast<int64_t>(params.p[i].tiles_n) * ((tasks[i].M + plan.tile[i].tm - 1) / plan.tile[i].tm);
    if (tiles * plan.splits > 0x7fffffff) return cudaErrorInvalidConfiguration;
  }
  const LaunchShape shape{dim3(static_cast<unsigned>(tiles * plan.splits)), kThreads, plan.splits, plan.smem_bytes};
  return launch_early(c.stream, shape, kern, params);
}

// What a product takes this way in tiles of `tm` rows of X with `splits` CTAs along K, in microseconds.
// Fitted to products of 1 to 1024 rows with the weights in the L2 cache (within 15 %; with weights
// from HBM calls of a few rows take 2 to 6 us more): a K block of 16 KB of weights takes a CTA 0.16
// us, more once X's tile outweighs the weight's (0.175 at 128 rows, 0.26 at 256), the gated form's two
// weights 0.22 to 0.25; the partial sums' way through shared memory 17 ns a row (gated: 25).
struct Cost {
  int64_t ctas;
  double per_cta;  // one CTA's time
  double feed;     // all SMs together take in at most 14 TB/s
};
Cost cost_of(const Task& t, int tm, int splits) {
  const bool gated = t.form == kGated;
  const int64_t blocks = (t.K + kBK - 1) / kBK * (t.form == kJoined ? 2 : 1);
  const int64_t tiles = (t.N + kTileN - 1) / kTileN * ((t.M + tm - 1) / tm);
  double block = tm <= 64 ? 0.16 : tm <= 128 ? 0.16 + (tm - 64) * 0.00023 : 0.175 + (tm - 128) * 0.00066;
  if (gated) block = 0.22 + tm * 0.00025;
  Cost c;
  c.ctas = tiles * splits;
  c.per_cta = static_cast<double>((blocks + splits - 1) / splits) * block + tm * (gated ? 0.025 : 0.017);
  c.feed = static_cast<double>(tiles) * static_cast<double>(blocks) *
           ((gated ? 2 : 1) * kWeightBytes + tm * kBK * 2) / 14e6;
  return c;
}

// SMs that clusters of `splits` CTAs reach when a CTA fills an SM: measured 152, 152, 144 and 120 of 152.
int reach_of(int splits, int sms) { return splits <= 2 ? sms : splits == 4 ? sms * 95 / 100 : sms * 79 / 100; }

}  // namespace

RowsPlan plan_rows(const Task* tasks, int n, int sms) {
  constexpr double kNextCta = 1.5, kNever = 1e30;
  RowsPlan plan;
  plan.cost = 0.0;
  bool one_wave = false;
  for (int splits = 1; splits <= kMaxSplits; splits *= 2) {
    const int reach = reach_of(splits, sms);
    int tm[kMaxProblems] = {};
    int64_t ctas = 0;
    double longest = 0.0, work = 0.0, feed = 0.0;
    bool too_long = false;
    for (int i = 0; i < n; ++i) {
      const Task& t = tasks[i];
      const int weights = t.form == kGated ? 2 : 1;
      const int64_t blocks = (t.K + kBK - 1) / kBK * (t.form == kJoined ? 2 : 1);
      if (splits > 1 && blocks < 2 * splits) {
        longest = -1.0;  // fewer than two blocks to a CTA
        break;
      }
      too_long = too_long || (blocks + splits - 1) / splits > kMaxPiece / kBK;
      // Equal shares of M: the fewest tiles that hold 256 sums per TMEM lane, or tiles of fewer rows.
      const int64_t fewest = (t.M * weights + 255) / 256;
      double best = 0.0;
      Cost chosen = {};
      for (const int rows : {256, 192, 128, 96, 64, 32}) {
        int64_t tiles_m = (t.M + rows - 1) / rows;
        if (tiles_m < fewest) tiles_m = fewest;
        const int candidate = static_cast<int>(((t.M + tiles_m - 1) / tiles_m + 15) / 16 * 16);
        if (candidate == tm[i]) continue;
        const Cost c = cost_of(t, candidate, splits);
        // Alone a product's waves count; among others, the SMs' time it takes.
        double time = n == 1 ? c.per_cta + static_cast<double>((c.ctas - 1) / reach) * (c.per_cta + kNextCta)
                             : (0.5 + static_cast<double>(c.ctas) / reach) * c.per_cta;
        if (time < c.feed) time = c.feed;
        if (best == 0.0 || time < best) {
          best = time;
          chosen = c;
          tm[i] = candidate;
        }
      }
      ctas += chosen.ctas;
      if (longest < chosen.per_cta) longest = chosen.per_cta;
      work += static_cast<double>(chosen.ctas) * chosen.per_cta;
      feed += chosen.feed;
    }
    if (longest < 0.0) break;
    if (plan.cost > 0.0 && ctas > 2 * reach) break;
    if (too_long) continue;
    // CTAs beyond the first on each SM: as long as the average, and their own start.
    const double average = work / static_cast<double>(ctas);
    double time = longest + static_cast<double>((ctas - 1) / reach) * (average + kNextCta);
    if (time < feed) time = feed;
    // What every launch takes, and a cluster's two barriers.
    time += 4.0 + (splits > 1 ? 0.6 : 0.0);
    if (plan.cost == 0.0 || time < plan.cost) {
      plan.cost = time;
      plan.splits = splits;
      for (int i = 0; i < n; ++i) plan.tile[i].tm = tm[i];
      one_wave = ctas <= reach;
    }
  }
  if (plan.cost == 0.0) {  // a CTA's sum would be longer than its accumulator takes
    plan.cost = kNever;
    return plan;
  }
  for (int i = 0; i < n; ++i) {
    const Task& t = tasks[i];
    RowsTile& tile = plan.tile[i];
    const int weights = t.form == kGated ? 2 : 1;
    const int x_bytes = t.A.k_major ? tile.tm * kBK * 2 : (tile.tm + 63) / 64 * kBoxBytes;
    tile.stage_bytes = static_cast<uint32_t>(weights * kWeightBytes + x_bytes);
    tile.tmem_cols = 32;
    while (tile.tmem_cols < static_cast<uint32_t>(weights * tile.tm)) tile.tmem_cols *= 2;
    // Half of an SM's memory where that holds six slots (then the next call's CTAs can be set up beside
    // these: linear 8x8192x4096 6 % shorter than with all of it) or more CTAs are to come; otherwise
    // a ring over all of it (64x4096x4096 3 % shorter than with half, 128x4096x4096 12 %).
    const int half = 112 * 1024, whole = 200 * 1024, stage = static_cast<int>(tile.stage_bytes);
    const int budget = !one_wave || 6 * stage <= half ? half : whole;
    // The partial sums lie over the ring, so it holds at least those.
    const int partials = weights * tile.tm * kTileN * 4;
    const int64_t blocks = (t.K + kBK - 1) / kBK * (t.form == kJoined ? 2 : 1);
    const int64_t per_cta = (blocks + plan.splits - 1) / plan.splits;
    int stages = budget / stage;
    if (stages > kMaxStages) stages = kMaxStages;
    if (stages > per_cta) stages = static_cast<int>(per_cta);
    const int least = (partials + stage - 1) / stage;
    if (stages < least) stages = least;
    tile.stages = stages;
    const int smem = stages * stage + 1024 + 512;
    if (plan.smem_bytes < smem) plan.smem_bytes = smem;
    // CTAs that share an SM must find TMEM for all of them, or clusters could wait for each other's:
    // shared memory in the proportion of TMEM (and never so little that a CTA fits beside a kernel
    // that fills the rest) keeps the sum of their columns at most 512.
    const int share = static_cast<int>(227 * 1024 * static_cast<int64_t>(tile.tmem_cols) / 512);
    if (plan.smem_bytes < share) plan.smem_bytes = share;
  }
  if (plan.smem_bytes < 48 * 1024) plan.smem_bytes = 48 * 1024;
  return plan;
}

cudaError_t run_rows(const Context& c, const Task* tasks, const RowsPlan& plan, int n) {
  if (n == 0) return cudaSuccess;
  const bool gated = tasks[0].form == kGated;
  if (c.kind == kBf16)
    return gated ? launch<kBf16, true>(c, tasks, plan, n) : launch<kBf16, false>(c, tasks, plan, n);
  return gated ? launch<kF16, true>(c, tasks, plan, n) : launch<kF16, false>(c, tasks, plan, n);
}

}  // namespace ff
}  // namespace t2s
