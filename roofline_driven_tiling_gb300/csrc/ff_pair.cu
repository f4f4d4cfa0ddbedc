// ff_pair.cu -- the products of the feed-forward operators on pairs of SMs (tcgen05 .cta_group::2).
//
// One persistent launch takes the tiles of up to three products (a gradient's dX and weight
// gradients run together, so that one product's last round is filled by the next one's tiles).
// A tile is 256 rows x up to 256 sums, computed by a cluster of two CTAs on two SMs: each
// stages its 128 rows of A and half of the columns of B (one 64-deep K block per ring slot), rank 0
// issues the MMAs, and each CTA's TMEM holds the sums of its 128 rows.
//
// Operands are read where they lie, whatever their order: rows along K (K-major boxes of 64
// values x rows) or K rows of outputs (MN-major boxes of 64 outputs x 64 K rows), both in
// 128-byte swizzle. That covers X W, dZ W^T and X^T dZ for weights of either order.
//
// What bounds it (sizes are rows x inputs x outputs, times those of the device in a captured graph with
// everything in the L2 cache that fits there): at large sizes the tensor cores under the power limit (8192^3
// 616-639 us, 1720-1785 TFLOP/s; torch.mm of the same size 590-634), with the last round of tiles on top
// (4096^3: 256 tiles on 76 pairs, 77 us on a GPU that was idle, 84-85 among other large products; with gelu_tanh,
// bias and saved pre-activations 82-92). Below about K = 1024 the epilogue: a 256 x 256 tile leaves the SM in about
// 2.2 us, 2.2 us more with gelu and 2 us more with a residual, against 0.26 us per K block (8192x256x2048
// 13.3 us, with gelu, bias and residual 30.5). A K block needs 64 bytes a clock into each SM, what its port
// takes; narrower tiles need more, so widths below 256 are for sizes that do not fill the pairs.
//
// A small weight's gradient over many rows has too few tiles for the pairs (1024 x 1024: 16), so its sum is
// cut into pieces along K: the pieces are tiles like any other, their FP32 sums go to the workspace (through
// L2) and a second launch adds them in their order. Gradients 32768x1024x256 with silu and db 133 -> 58 us,
// gated 65536x512x512 218 -> 150, 16384x1024x1024 130 -> 115-118 (floor of both 72).
//
// Two accumulators of 256 columns fill TMEM, so a tile's epilogue runs under the next tile's MMAs.
// Six ring slots of 32 KB leave 35 KB for the epilogue's boxes; five cost 1.5 % at 4096^3.
//
// An accumulator takes at most kMaxPiece values of K (its truncation grows with them). A tile of more
// sums them in turn into the two accumulators, and the epilogue's warps add each piece in FP32 to what the
// ones before it left in the other accumulator, which then takes the piece after it. The sums of a weight's
// gradient are cut over the SMs besides, as above.
//
// The gated product needs no wider machinery: rank 0 stages 128 columns of Wg and rank 1 the same
// 128 columns of Wu, so the lower half of the accumulator's columns holds G, the upper half U.
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

constexpr int kRows = 128;    // A rows of one CTA
constexpr int kStages = 6;    // ring slots of 32 KB (narrow tiles: four of 48 KB)
constexpr int kMaxN = 256;    // widest MMA
constexpr int kABytes = kRows * kBK * 2;
constexpr int kBBytes = kMaxN / 2 * kBK * 2;
constexpr int kStageBytes = kABytes + kBBytes;
// Tiles of up to 128 columns take two K blocks per slot: a slot's waits, commit and copies take longer to issue
// than a narrow block's MMAs take to run (a K block of 128 columns 0.20 -> 0.17 us, of 64 0.19 -> 0.16;
// 512x4096x4096 15 % shorter, 256x8192x8192 13 % with the widths chosen accordingly).
constexpr int kNarrowN = 128;
constexpr int kNarrowStages = 4;
constexpr int kNarrowStageBytes = 2 * (kABytes + kBoxBytes);
static_assert(kNarrowStages * kNarrowStageBytes <= kStages * kStageBytes, "the ring");
constexpr int kEpiWarps = 8;
constexpr int kThreads = 128 + 32 * kEpiWarps;
constexpr int kUnit = 32;                        // columns an epilogue warp takes at a time
constexpr int kUnitBytes = 32 * kUnit * 2;       // 32 rows of 64 bytes
constexpr int kStagingBytes = kEpiWarps * 2 * kUnitBytes;
constexpr int kBiasBytes = kEpiWarps * kUnit * 4;
constexpr int kSmemBytes = kStages * kStageBytes + 1024 + 1024 + kStagingBytes + kBiasBytes;
static_assert(kMaxN / (2 * kUnit) == 4, "column groups of an epilogue warp");
static_assert(kSmemBytes <= 227 * 1024, "shared memory of one CTA");
constexpr uint32_t kTmemCols = 512;  // two accumulators of 256 columns

struct PairProblem {
  CUtensorMap a[2], b[2], y, z, z2;
  const uint16_t* bias;
  const uint16_t* R;
  uint16_t *Y, *Z, *Z2;
  int64_t ldr, ldy, ldz, ldz2;
  int M, N;
  int nkb, nkb_first;  // ring slots of K, and how many of them come from a[0], b[0]
  int tiles_m, tiles_n;
  int splits, split_blocks;  // pieces of the sum over K, and their slots (the last: the rest)
  int acc_blocks;            // slots that one accumulator takes
  float* partials;           // of the pieces' sums; nullptr: one piece, stored through the epilogue
  int bn;       // columns of Y in a tile
  int mma_n;    // sums per row in a tile (gated: 2 bn)
  uint32_t idesc;
  uint32_t stage_tx;  // bytes that both CTAs copy per slot
  int a_k_major, b_k_major, b_boxes;
  int y_tma, z_tma, z2_tma, r_wide;
  int act;
};

struct PairParams {
  PairProblem p[kMaxProblems];
  int first[kMaxProblems + 1];  // first tile of each problem; the last entry is the tile count
  int narrow;                   // two K blocks per slot
  unsigned* status;
};

// Column groups of 8 tile rows sweep the columns together, so that the tiles in flight share A
// and B in the L2 cache.
__device__ __forceinline__ void tile_at(const PairProblem& p, int t, int& m0, int& n0) {
  tc::tile_origin(t, p.tiles_m, p.tiles_n, 2 * kRows, p.bn, m0, n0);
}

// The slots of K of a piece of the sum; pieces of the same slots follow each other in the tile order.
struct Piece {
  int tile, first, blocks;
};
template <bool SPLIT>
__device__ __forceinline__ Piece piece_at(const PairProblem& p, int t) {
  if (!SPLIT || p.splits == 1) return {t, 0, p.nkb};
  const int tiles = p.tiles_m * p.tiles_n, piece = t / tiles, first = piece * p.split_blocks;
  return {t - piece * tiles, first, min(p.split_blocks, p.nkb - first)};
}

__device__ __forceinline__ void ld_shared_v4(uint32_t addr, uint32_t (&v)[4]) {
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3])
               : "r"(addr));
}

// Byte offset of 16-byte chunk `c` of row `r` in a 32 x 64-byte box (64-byte swizzle).
__device__ __forceinline__ uint32_t unit_chunk(int r, int c) {
  return static_cast<uint32_t>(r) * 64u + (static_cast<uint32_t>(c ^ ((r >> 1) & 3)) << 4);
}

// One epilogue warp's two staging boxes, taken in turn.
struct Staging {
  uint32_t base;
  uint32_t count;
  int lane;

  // The next box, free of the TMA store that last used it.
  __device__ __forceinline__ uint32_t next() {
    const uint32_t at = base + (count++ & 1u) * kUnitBytes;
    if (lane == 0) bulk_wait_read_but_one();
    __syncwarp();
    return at;
  }
};

// Stores a warp's 32 x 32 outputs at (m, n) from its box, each lane having written its own row:
// by TMA, or (rows not 16-byte aligned) one row of 32 values per instruction.
__device__ __forceinline__ void store_unit(const CUtensorMap* map, bool tma, uint32_t box, uint16_t* p, int64_t ld,
                                           int m, int n, int M, int N, int lane) {
  if (tma) {
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) tma_store_2d(map, box, n, m);
    return;
  }
  __syncwarp();
  // Eight rows at a time; the swizzle of row 8 g + j is that of row j.
  uint32_t from[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) from[i] = box + (static_cast<uint32_t>((lane >> 3) ^ i) << 4) + (lane & 7) * 2;
  uint16_t* out = p + static_cast<int64_t>(m) * ld + n + lane;
  const int rows = n + lane < N ? M - m : 0;
#pragma unroll 1
  for (int r = 0; r < 32; r += 8) {
    uint16_t v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j)
      asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v[j]) : "r"(from[j >> 1] + static_cast<uint32_t>(r + j) * 64u));
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if (r + j < rows) *out = v[j];
      out += ld;
    }
  }
  __syncwarp();
  // The TMA-store count that next() waits by: an empty group stands for this box.
  if (lane == 0) asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}

// The residual's 32 x 32 values at (m, n), zeros outside the matrix: fetched four lanes to a row of 64
// bytes, some time before they are placed in the box; or (rows not 16-byte aligned, or cut by the
// matrix's edge) read into the box value by value.
struct Residual {
  uint4 v[4];
  bool fetched;

  __device__ __forceinline__ void fetch(const PairProblem& p, int m, int n, int lane) {
    fetched = p.R != nullptr && p.r_wide && n + kUnit <= p.N && m < p.M;
    if (!fetched) return;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = m + 8 * i + (lane >> 2);
      v[i] = make_uint4(0, 0, 0, 0);
      if (r < p.M) v[i] = *reinterpret_cast<const uint4*>(p.R + static_cast<int64_t>(r) * p.ldr + n + (lane & 3) * 8);
    }
  }
  __device__ __forceinline__ void place(const PairProblem& p, uint32_t box, int m, int n, int lane) const {
    if (fetched) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        st_shared_v4(box + unit_chunk(8 * i + (lane >> 2), lane & 3), v[i].x, v[i].y, v[i].z, v[i].w);
    } else {
#pragma unroll 8
      for (int r = 0; r < 32; ++r) {
        uint16_t x = 0;
        if (m + r < p.M && n + lane < p.N) x = p.R[static_cast<int64_t>(m + r) * p.ldr + n + lane];
        asm volatile("st.shared.u16 [%0], %1;" ::"r"(box + unit_chunk(r, lane >> 3) + (lane & 7) * 2), "h"(x)
                     : "memory");
      }
    }
    __syncwarp();
  }
};

// A lane's row of 32 values, rounded, into the box.
template <int KIND>
__device__ __forceinline__ void put_row(uint32_t box, int lane, const uint64_t (&v)[kUnit / 2]) {
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = halves(v[4 * c + i]);
      w[i] = pack_f32<KIND>(f.x, f.y);
    }
    st_shared_v4(box + unit_chunk(lane, c), w[0], w[1], w[2], w[3]);
  }
}

// Loaded accumulator columns as sums; of no K block, zeros.
__device__ __forceinline__ void sums_of(const uint32_t (&r)[kUnit], bool any, uint64_t (&s)[kUnit / 2]) {
#pragma unroll
  for (int i = 0; i < kUnit / 2; ++i)
    s[i] = any ? pack2(__uint_as_float(r[2 * i]), __uint_as_float(r[2 * i + 1])) : 0ull;
}

// Adds one accumulator's 32 columns of the warp's 32 rows to another's.
__device__ __forceinline__ void add_columns(uint32_t to, uint32_t from) {
#pragma unroll
  for (uint32_t c = 0; c < kUnit; c += 16) {
    uint32_t x[16], y[16];
    tc::tmem_ld16(to + c, x);
    tc::tmem_ld16(from + c, y);
#pragma unroll
    for (int i = 0; i < 16; ++i) asm volatile("" : "+r"(x[i]), "+r"(y[i]));  // no use before the loads' waits
#pragma unroll
    for (int i = 0; i < 16; ++i) x[i] = __float_as_uint(__uint_as_float(y[i]) + __uint_as_float(x[i]));
    store_columns16(to + c, x);
  }
}

// Roles: warps 0 and 2 copy A and B, warp 1 issues the MMAs (rank 0 only), warps 4..11 are the
// epilogue (warp 3 only holds TMEM). full[s] / empty[s] per ring slot, acc_full[b] / acc_empty[b] per accumulator; a role
// that gives up a bounded wait records it and stops, and the others' own waits end the same way.
// LONG: some tile's sum takes more than one accumulator.
template <int KIND, bool GATED, bool SPLIT, bool LONG>
__global__ void __launch_bounds__(kThreads, 1) ff_pair_kernel(const __grid_constant__ PairParams params) {
  extern __shared__ uint8_t smem_raw[];
  const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
  const uint32_t bars = base + kStages * kStageBytes;
  auto full = [&](int s) { return bars + 8u * s; };
  auto empty = [&](int s) { return bars + 8u * (kStages + s); };
  const uint32_t acc_full = bars + 16u * kStages, acc_empty = acc_full + 16u, mma_done = acc_empty + 16u;
  const uint32_t slot = mma_done + 8u;
  const uint32_t staging = bars + 1024u;
  unsigned* const status = params.status;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = static_cast<int>(cluster_ctarank());
  const int tile0 = static_cast<int>(cluster_id_x()), tile_step = static_cast<int>(cluster_count_x());
  const int tiles = params.first[kMaxProblems];
  const bool narrow = params.narrow != 0;
  const int stages = narrow ? kNarrowStages : kStages;
  const uint32_t stage_bytes = narrow ? kNarrowStageBytes : kStageBytes, b_offset = narrow ? 2 * kABytes : kABytes;
  auto problem_of = [&](int t) { return t < params.first[1] ? 0 : t < params.first[2] ? 1 : 2; };

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
  if (warp == 0 && elect_one()) tma_prefetch_desc(&params.p[0].a[0]);
  if (warp == 2 && elect_one()) tma_prefetch_desc(&params.p[0].b[GATED ? rank : 0]);
  if (warp == 3) tc::tmem_alloc<2>(slot, kTmemCols);
  tc::tc_fence_before();
  __syncthreads();
  cluster_sync_all();  // the peer's copies and commits arrive on these barriers
  wait_for_earlier_kernels();
  tc::tc_fence_after();
  uint32_t tmem;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(tmem) : "r"(slot) : "memory");

  if (warp == 0 || warp == 2) {
    // Copies of A (warp 0) and of B (warp 2): a warp each, so that neither's instructions
    // between two copies hold up the other's.
    {
      const bool is_a = warp == 0;
      Ring ring(base + (is_a ? 0 : b_offset), stage_bytes, full(0), empty(0), stages, narrow ? 2 * kBK : kBK);
      const uint32_t second = narrow ? (is_a ? kABytes : kBoxBytes) : 0u;  // where a slot's second K block lies
      const uint32_t bar0 = tc::map_to_rank(full(0), 0);  // both CTAs' copies complete on rank 0's
      const bool expects = is_a && rank == 0;
      bool ok = true;
      for (int t = tile0; ok && t < tiles; t += tile_step) {
        const int pi = problem_of(t);
        const PairProblem& p = params.p[pi];
        const Piece piece = piece_at<SPLIT>(p, t - params.first[pi]);
        int m0, n0;
        tile_at(p, piece.tile, m0, n0);
        // Gated: the same columns of this rank's weight; otherwise this rank's half of them.
        const int at = is_a ? m0 + rank * kRows : GATED ? n0 : n0 + rank * (p.mma_n / 2);
        const bool k_major = is_a ? p.a_k_major : p.b_k_major;
        const int boxes = is_a ? kRows / 64 : p.b_boxes;
        const uint32_t bytes = p.stage_tx;
        int from = piece.first, to = SPLIT ? min(p.nkb_first, from + piece.blocks) : p.nkb_first;
        int left = from + piece.blocks - to;
        const CUtensorMap* map = is_a ? &p.a[0] : &p.b[GATED ? rank : 0];
        while (ok) {
          if (k_major) {
            ok = ring.copy(from, to, expects ? bytes : 0u, bar0, status, [&](uint32_t st, int k0, uint32_t bar) {
              tc::tma_load_2d_pair(st, map, k0, at, bar);
              if (second != 0) tc::tma_load_2d_pair(st + second, map, k0 + kBK, at, bar);
            });
          } else if (boxes > 1) {
            ok = ring.copy(from, to, expects ? bytes : 0u, bar0, status, [&](uint32_t st, int k0, uint32_t bar) {
              tc::tma_load_2d_pair(st, map, at, k0, bar);
              tc::tma_load_2d_pair(st + kBoxBytes, map, at + 64, k0, bar);
              if (second != 0) {
                tc::tma_load_2d_pair(st + second, map, at, k0 + kBK, bar);
                tc::tma_load_2d_pair(st + second + kBoxBytes, map, at + 64, k0 + kBK, bar);
              }
            });
          } else {
            ok = ring.copy(from, to, expects ? bytes : 0u, bar0, status, [&](uint32_t st, int k0, uint32_t bar) {
              tc::tma_load_2d_pair(st, map, at, k0, bar);
              if (second != 0) tc::tma_load_2d_pair(st + second, map, at, k0 + kBK, bar);
            });
          }
          if (left == 0) break;
          from = 0;
          to = left;
          left = 0;
          map = is_a ? &p.a[1] : &p.b[1];
        }
      }
      // Every slot's copies have landed and been read before the CTA may go.
      if (ok) ring.copy(0, stages, 0u, bar0, status, [](uint32_t, int, uint32_t) {});
    }
  } else if (warp == 1) {
    if (rank == 0) {
      int s = 0, use = 0;
      uint32_t phase = 0, st = base;
      bool ok = true;
      for (int t = tile0; ok && t < tiles; t += tile_step) {
        const int pi = problem_of(t);
        const PairProblem& p = params.p[pi];
        const OperandForm fa = operand_form(p.a_k_major), fb = operand_form(p.b_k_major);
        const uint32_t idesc = p.idesc;
        const int nkb = piece_at<SPLIT>(p, t - params.first[pi]).blocks;
        int left = nkb;
        do {
          const int blocks = LONG ? min(left, p.acc_blocks) : nkb, b = use & 1;
          const uint32_t acc = tmem + static_cast<uint32_t>(b) * kMaxN;
          if (!__all_sync(0xffffffffu, wait_bounded(acc_empty + 8u * b, ((use >> 1) & 1u) ^ 1u, status))) {
            ok = false;
            break;
          }
          tc::tc_fence_after();
#pragma unroll 1
          for (int kb = 0; kb < blocks; ++kb) {
            const uint64_t da = with_address(fa, st), db = with_address(fb, st + b_offset);
            if (!__all_sync(0xffffffffu, wait_bounded(full(s), phase, status))) {
              ok = false;
              break;
            }
            tc::tc_fence_after();
            mma_block<2>(acc, da, fa.step, db, fb.step, idesc, kb);
            if (narrow) mma_block<2>(acc, da + (kABytes >> 4), fa.step, db + (kBoxBytes >> 4), fb.step, idesc, 1u);
            if (elect_one()) tc::mma_commit_pair(empty(s));
            __syncwarp();
            st += stage_bytes;
            if (++s == stages) {
              s = 0;
              st = base;
              phase ^= 1u;
            }
          }
          if (ok && elect_one()) tc::mma_commit_pair(acc_full + 8u * b);
          __syncwarp();
          ++use;
          left -= blocks;
        } while (LONG && ok && left > 0);
      }
      // Every MMA issued above ends before TMEM is released.
      if (elect_one()) tc::mma_commit<2>(mma_done);
      __syncwarp();
      wait_bounded(mma_done, 0u, status);
    }
  } else if (warp >= 4) {
    const int e = warp - 4, q = warp & 3, half = e >> 2;
    Staging boxes{staging + static_cast<uint32_t>(e) * 2u * kUnitBytes, 0u, lane};
    const uint32_t bias_row = staging + kStagingBytes + static_cast<uint32_t>(e) * kUnit * 4u;
    int use = 0;
    for (int t = tile0; t < tiles; t += tile_step, ++use) {
      const int pi = problem_of(t);
      const PairProblem& p = params.p[pi];
      const Piece piece = piece_at<SPLIT>(p, t - params.first[pi]);
      int m0, n0;
      tile_at(p, piece.tile, m0, n0);
      const int m = m0 + rank * kRows + 32 * q;
      // What the epilogue reads from memory is on its way before the sums are there: the bias of
      // this warp's columns (lane i has column i of each group of 32) and the first residual box.
      Residual residual;
      float bias[kMaxN / (2 * kUnit)] = {};
      if (!GATED) {
        residual.fetch(p, m, n0 + half * kUnit, lane);
        if (p.bias != nullptr) {
#pragma unroll
          for (int i = 0; i < kMaxN / (2 * kUnit); ++i) {
            const int c = (2 * i + half) * kUnit + lane;
            if (c < p.bn && n0 + c < p.N) bias[i] = to_f32<KIND>(p.bias[n0 + c]);
          }
        }
      }
      // The two warps of a row quarter take every other group of 32 columns inside the matrix; a
      // group's sums are on their way from TMEM while the one before it is stored.
      const int columns = m < p.M ? min(p.bn, p.N - n0) : 0;
      const uint32_t rows_at = tmem + (static_cast<uint32_t>(32 * q) << 16);
      bool done = __all_sync(0xffffffffu, wait_bounded(acc_full + 8u * (use & 1), (use >> 1) & 1u, status));
      if constexpr (LONG) {
        for (int left = piece.blocks - p.acc_blocks; done && left > 0; left -= p.acc_blocks) {
          const uint32_t before = static_cast<uint32_t>(use & 1);
          ++use;
          done = __all_sync(0xffffffffu, wait_bounded(acc_full + 8u * (use & 1), (use >> 1) & 1u, status));
          if (!done) break;
          tc::tc_fence_after();
          for (int c = half * kUnit; c < columns; c += 2 * kUnit) {
            add_columns(rows_at + (before ^ 1u) * kMaxN + c, rows_at + before * kMaxN + c);
            if (GATED) add_columns(rows_at + (before ^ 1u) * kMaxN + p.bn + c, rows_at + before * kMaxN + p.bn + c);
          }
          wait_stored_columns();
          tc::tc_fence_before();
          __syncwarp();
          if (lane == 0) arrive_remote(tc::map_to_rank(acc_empty + 8u * before, 0));
        }
      }
      if (!done) break;
      tc::tc_fence_after();
      const int b = use & 1;
      const uint32_t acc = rows_at + static_cast<uint32_t>(b) * kMaxN;
      const bool any = p.nkb > 0;
      uint32_t sums[kUnit], gated_sums[GATED ? kUnit : 1];
      auto load = [&](int c) {
        load_columns(acc + static_cast<uint32_t>(c), sums);
        if constexpr (GATED) load_columns(acc + static_cast<uint32_t>(p.bn + c), gated_sums);
      };
      if (half * kUnit < columns) load(half * kUnit);
      for (int c = half * kUnit; c < columns; c += 2 * kUnit) {
        const int n = n0 + c;
        const bool more = c + 2 * kUnit < columns;
        uint64_t v[kUnit / 2];
        wait_columns(sums);
        sums_of(sums, any, v);
        if constexpr (GATED) {
          uint64_t u[kUnit / 2];
          wait_columns(gated_sums);
          sums_of(gated_sums, any, u);
          if (p.Z != nullptr) {
            const uint32_t box = boxes.next();
            put_row<KIND>(box, lane, v);
            store_unit(&p.z, p.z_tma, box, p.Z, p.ldz, m, n, p.M, p.N, lane);
          }
          if (p.Z2 != nullptr) {
            const uint32_t box = boxes.next();
            put_row<KIND>(box, lane, u);
            store_unit(&p.z2, p.z2_tma, box, p.Z2, p.ldz2, m, n, p.M, p.N, lane);
          }
          with_act(p.act, [&](auto a) {
#pragma unroll
            for (int i = 0; i < kUnit / 2; ++i) v[i] = mul2(act_pair<decltype(a)::value>(v[i]), u[i]);
          });
          const uint32_t box = boxes.next();
          put_row<KIND>(box, lane, v);
          if (more) load(c + 2 * kUnit);
          store_unit(&p.y, p.y_tma, box, p.Y, p.ldy, m, n, p.M, p.N, lane);
        } else if (SPLIT && p.partials != nullptr) {
          // Four columns of 256 rows together, so that a warp's store is 512 bytes in a row.
          float4* out = reinterpret_cast<float4*>(p.partials) +
                        (static_cast<int64_t>(t - params.first[pi]) * p.bn + c) / 4 * (2 * kRows) + rank * kRows + 32 * q + lane;
#pragma unroll
          for (int i = 0; i < kUnit / 4; ++i) {
            const float2 lo = halves(v[2 * i]), hi = halves(v[2 * i + 1]);
            out[i * 2 * kRows] = make_float4(lo.x, lo.y, hi.x, hi.y);
          }
          if (more) load(c + 2 * kUnit);
        } else {
          if (p.bias != nullptr) {
            const int i = c / (2 * kUnit);
            const float mine = i == 0 ? bias[0] : i == 1 ? bias[1] : i == 2 ? bias[2] : bias[3];
            __syncwarp();
            asm volatile("st.shared.f32 [%0], %1;" ::"r"(bias_row + 4u * lane), "f"(mine) : "memory");
            __syncwarp();
#pragma unroll
            for (int i = 0; i < kUnit; i += 4) {
              uint64_t lo, hi;
              lds128_pairs(bias_row + 4u * i, lo, hi);
              v[i / 2] = add2(v[i / 2], lo);
              v[i / 2 + 1] = add2(v[i / 2 + 1], hi);
            }
          }
          if (p.Z != nullptr) {
            const uint32_t box = boxes.next();
            put_row<KIND>(box, lane, v);
            store_unit(&p.z, p.z_tma, box, p.Z, p.ldz, m, n, p.M, p.N, lane);
          }
          with_act(p.act, [&](auto a) {
#pragma unroll
            for (int i = 0; i < kUnit / 2; ++i) v[i] = act_pair<decltype(a)::value>(v[i]);
          });
          const uint32_t box = boxes.next();
          if (p.R != nullptr) {
            residual.place(p, box, m, n, lane);
            if (more) residual.fetch(p, m, n + 2 * kUnit, lane);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              uint32_t r[4];
              ld_shared_v4(box + unit_chunk(lane, i), r);
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                const float2 x = to_f32x2<KIND>(r[j]);
                v[4 * i + j] = add2(v[4 * i + j], pack2(x.x, x.y));
              }
            }
          }
          put_row<KIND>(box, lane, v);
          if (more) load(c + 2 * kUnit);
          store_unit(&p.y, p.y_tma, box, p.Y, p.ldy, m, n, p.M, p.N, lane);
        }
      }
      tc::tc_fence_before();
      __syncwarp();
      if (lane == 0) arrive_remote(tc::map_to_rank(acc_empty + 8u * b, 0));
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

// Adds the pieces' sums in their order. A block takes eight columns of a tile's 256 rows.
struct PieceSums {
  const float4* partials[kMaxProblems];
  uint16_t* Y[kMaxProblems];
  int64_t ldy[kMaxProblems];
  int M[kMaxProblems], N[kMaxProblems], tiles_m[kMaxProblems], tiles_n[kMaxProblems], splits[kMaxProblems];
  int wide[kMaxProblems];
  unsigned first[kMaxProblems + 1];  // first block of each
  int bn;
};

template <int KIND>
__global__ void __launch_bounds__(2 * kRows) piece_sum_kernel(const __grid_constant__ PieceSums s) {
  wait_for_earlier_kernels();
  const int i = blockIdx.x < s.first[1] ? 0 : blockIdx.x < s.first[2] ? 1 : 2;
  const int chunks = s.bn / 8, unit = static_cast<int>(blockIdx.x - s.first[i]), tile = unit / chunks;
  int m0, n0;
  tc::tile_origin(tile, s.tiles_m[i], s.tiles_n[i], 2 * kRows, s.bn, m0, n0);
  const int m = m0 + static_cast<int>(threadIdx.x), n = n0 + (unit - tile * chunks) * 8;
  if (m >= s.M[i] || n >= s.N[i]) return;
  const int64_t step = static_cast<int64_t>(s.tiles_m[i]) * s.tiles_n[i] * (s.bn / 4) * (2 * kRows);
  const float4* from = s.partials[i] + static_cast<int64_t>(unit) * 2 * (2 * kRows) + threadIdx.x;
  float4 lo = make_float4(0.0f, 0.0f, 0.0f, 0.0f), hi = lo;
  constexpr int kAhead = 8;  // pieces on their way before the first is added (four: 0.5 to 3 us slower)
  for (int j = 0; j < s.splits[i]; j += kAhead) {
    float4 a[kAhead], b[kAhead];
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      a[k] = b[k] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      if (j + k < s.splits[i]) {
        a[k] = from[0];
        b[k] = from[2 * kRows];
        from += step;
      }
    }
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      lo.x += a[k].x, lo.y += a[k].y, lo.z += a[k].z, lo.w += a[k].w;
      hi.x += b[k].x, hi.y += b[k].y, hi.z += b[k].z, hi.w += b[k].w;
    }
  }
  const uint32_t w[4] = {pack_f32<KIND>(lo.x, lo.y), pack_f32<KIND>(lo.z, lo.w), pack_f32<KIND>(hi.x, hi.y),
                         pack_f32<KIND>(hi.z, hi.w)};
  uint16_t* y = s.Y[i] + m * s.ldy[i] + n;
  if (s.wide[i] && n + 8 <= s.N[i]) {
    *reinterpret_cast<uint4*>(y) = make_uint4(w[0], w[1], w[2], w[3]);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (n + j < s.N[i]) y[j] = static_cast<uint16_t>(w[j / 2] >> 16 * (j & 1));
  }
}

// Resident clusters of a kernel on the current device, looked up once.
template <int KIND, bool GATED, bool SPLIT, bool LONG>
cudaError_t resident_clusters(int* out) {
  constexpr int kMaxDevices = 64;
  static std::atomic<int> known[kMaxDevices];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
  int n = known[dev].load(std::memory_order_acquire);
  if (n == 0) {
    auto kern = ff_pair_kernel<KIND, GATED, SPLIT, LONG>;
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

// The store map of an output, where its rows allow one: on 16-byte boundaries and of whole 16-byte
// words (a store clipped at an odd width still writes the whole of its last 16 bytes).
cudaError_t output_map(CUtensorMap* m, int* usable, const Matrix& o, int64_t M, int64_t N) {
  *usable = 0;
  if (o.p == nullptr || N % 8 != 0 || !aligned16(o.p, o.ld)) return cudaSuccess;
  *usable = 1;
  return encode_tmap_16bit_2d(m, o.p, N, M, o.ld, kUnit, 32, CU_TENSOR_MAP_SWIZZLE_64B);
}

// K values of a ring slot.
int slot_depth(int width) { return width <= kNarrowN ? 2 * kBK : kBK; }

template <int KIND>
cudaError_t fill(PairProblem* p, const Task& t, int mma_n, int splits) {
  const bool gated = t.form == kGated;
  cudaError_t e = cudaSuccess;
  p->M = static_cast<int>(t.M);
  p->N = static_cast<int>(t.N);
  p->mma_n = mma_n;
  p->bn = gated ? mma_n / 2 : mma_n;
  if (p->bn % kUnit != 0) return cudaErrorInvalidValue;
  p->tiles_m = static_cast<int>((t.M + 2 * kRows - 1) / (2 * kRows));
  p->tiles_n = static_cast<int>((t.N + p->bn - 1) / p->bn);
  // A narrow tile's last slot may reach past K: its copies read zeros there.
  const int depth = slot_depth(mma_n);
  const int blocks = static_cast<int>((t.K + depth - 1) / depth);
  p->nkb_first = blocks;
  p->nkb = t.form == kJoined ? 2 * blocks : blocks;
  p->splits = 1;
  p->split_blocks = p->nkb;
  if (t.split && splits > 1) {
    p->split_blocks = (blocks + splits - 1) / splits;
    p->splits = (blocks + p->split_blocks - 1) / p->split_blocks;
  }
  p->acc_blocks = static_cast<int>(kMaxPiece) / depth;
  p->a_k_major = t.A.k_major;
  p->b_k_major = t.B.k_major;
  p->b_boxes = (mma_n / 2 + 63) / 64;
  const uint32_t b_bytes = p->b_k_major ? static_cast<uint32_t>(mma_n / 2) * kBK * 2
                                        : static_cast<uint32_t>(p->b_boxes) * kBoxBytes;
  p->stage_tx = static_cast<uint32_t>(2 * (depth / kBK)) * (kABytes + b_bytes);
  // D FP32, A and B of the 16-bit type, their orders, N and M = 256.
  const uint32_t fmt = KIND == kBf16 ? 1u : 0u;
  p->idesc = (1u << 4) | (fmt << 7) | (fmt << 10) | ((p->a_k_major ? 0u : 1u) << 15) |
             ((p->b_k_major ? 0u : 1u) << 16) | (static_cast<uint32_t>(mma_n >> 3) << 17) |
             (static_cast<uint32_t>(2 * kRows >> 4) << 24);
  p->bias = t.bias;
  p->R = t.R.p;
  p->ldr = t.R.ld;
  p->r_wide = t.R.p != nullptr && aligned16(t.R.p, t.R.ld);
  p->Y = t.Y.p;
  p->ldy = t.Y.ld;
  p->Z = t.Z.p;
  p->ldz = t.Z.ld;
  p->Z2 = t.Z2.p;
  p->ldz2 = t.Z2.ld;
  p->act = t.act;
  if (blocks > 0) {
    const uint32_t half = static_cast<uint32_t>(mma_n / 2);
    if ((e = operand_map(&p->a[0], t.A, t.M, t.K, kRows)) != cudaSuccess) return e;
    if ((e = operand_map(&p->b[0], t.B, t.N, t.K, half)) != cudaSuccess) return e;
    if (t.form == kJoined && (e = operand_map(&p->a[1], t.A2, t.M, t.K, kRows)) != cudaSuccess) return e;
    if (t.form != kLinear && (e = operand_map(&p->b[1], t.B2, t.N, t.K, half)) != cudaSuccess) return e;
  }
  if ((e = output_map(&p->y, &p->y_tma, t.Y, t.M, t.N)) != cudaSuccess) return e;
  if ((e = output_map(&p->z, &p->z_tma, t.Z, t.M, t.N)) != cudaSuccess) return e;
  return output_map(&p->z2, &p->z2_tma, t.Z2, t.M, t.N);
}

template <int KIND, bool GATED, bool SPLIT, bool LONG>
cudaError_t launch(const Context& c, const Task* tasks, const PairPlan& plan, int n) {
  int resident = 0;
  cudaError_t e = resident_clusters<KIND, GATED, SPLIT, LONG>(&resident);
  if (e != cudaSuccess) return e;
  PairParams params;
  memset(&params, 0, sizeof(params));
  params.status = c.status;
  params.narrow = plan.width <= kNarrowN;
  PieceSums sums;
  memset(&sums, 0, sizeof(sums));
  sums.bn = plan.width;
  int64_t tiles = 0, blocks = 0;
  size_t used = 0;
  for (int i = 0; i < kMaxProblems; ++i) {
    params.first[i] = static_cast<int>(tiles);
    sums.first[i] = static_cast<unsigned>(blocks);
    if (i >= n) continue;
    PairProblem& p = params.p[i];
    if ((e = fill<KIND>(&p, tasks[i], plan.width, plan.splits)) != cudaSuccess) return e;
    const int64_t outputs = static_cast<int64_t>(p.tiles_m) * p.tiles_n, pieces = outputs * p.splits;
    tiles += pieces;
    if (tiles > 0x7fffffff) return cudaErrorInvalidConfiguration;
    if (p.splits == 1) continue;
    p.partials = c.partials + used / 4;
    used += static_cast<size_t>(pieces) * 2 * kRows * p.bn * 4;
    if (used > c.partial_bytes) return cudaErrorInvalidConfiguration;
    sums.partials[i] = reinterpret_cast<const float4*>(p.partials);
    sums.Y[i] = p.Y, sums.ldy[i] = p.ldy;
    sums.M[i] = p.M, sums.N[i] = p.N;
    sums.tiles_m[i] = p.tiles_m, sums.tiles_n[i] = p.tiles_n, sums.splits[i] = p.splits;
    sums.wide[i] = aligned16(p.Y, p.ldy);
    blocks += outputs * (p.bn / 8);
  }
  sums.first[kMaxProblems] = static_cast<unsigned>(blocks);
  params.first[kMaxProblems] = static_cast<int>(tiles);
  const LaunchShape shape{dim3(static_cast<unsigned>(2 * (tiles < resident ? tiles : resident))), kThreads, 2, kSmemBytes};
  e = launch_early(c.stream, shape, ff_pair_kernel<KIND, GATED, SPLIT, LONG>, params);
  if (!SPLIT || e != cudaSuccess || blocks == 0) return e;
  return launch_early(c.stream, {dim3(static_cast<unsigned>(blocks)), 2 * kRows, 1, 0}, piece_sum_kernel<KIND>, sums);
}

}  // namespace

// Fitted to products of 256 to 4096 rows (most within 10 %): a K block takes a pair of SMs 0.158 us
// or the time of its MMAs and copies, whichever is longer, and a tile that others follow 0.3 us more;
// all SMs together compute 1.8 PFLOP/s (the power limit) and take in 16 TB/s; starting up, and a last
// tile's epilogue, take the rest.
PairPlan plan_pair(const Task* tasks, int n, int pairs, size_t partial_bytes) {
  struct Width {
    int n;
    double block;
  };
  static constexpr Width kWidths[] = {{64, 0.158}, {128, 0.17}, {192, 0.215}, {224, 0.235}, {256, 0.26}};
  // Pieces of a sum have eight K blocks at least (their stores take as long as four), and there is room
  // for them. Adding the pieces is a launch more, and their way through the L2 cache: fitted to dW of 256^2
  // to 1024^2 weights from 4096 to 65536 rows in 2 to 19 pieces (most within 10 %).
  constexpr int kLeastBlocks = 8;
  constexpr double kSumLaunch = 1.2, kSumPiece = 0.03;
  constexpr double kNextTile = 0.3, kCutTile = 0.8;  // a tile that others follow, and a piece with its stores
  PairPlan plan;
  int64_t longest = 0;
  for (int i = 0; i < n; ++i)
    if (tasks[i].split && longest < tasks[i].K) longest = tasks[i].K;
  const int64_t most_splits = partial_bytes > 0 ? longest / (kLeastBlocks * kBK) : 1;

  // The tiles of one width, and what no number of pieces makes shorter.
  struct Way {
    int width;
    double block, least;
    int64_t tiles[kMaxProblems], blocks[kMaxProblems], cut_tiles, cut_blocks;
    double whole_work, cut_work;  // SM pairs' time for the products that stay whole, and that are cut
  };
  Way ways[sizeof(kWidths) / sizeof(kWidths[0])];
  int n_ways = 0;
  for (const Width& w : kWidths) {
    Way& way = ways[n_ways];
    way.width = w.n, way.block = w.block;
    way.cut_tiles = way.cut_blocks = 0;
    way.whole_work = way.cut_work = 0.0;
    double flops = 0.0, bytes = 0.0;
    bool whole = true;
    for (int i = 0; i < n; ++i) {
      const Task& t = tasks[i];
      const int bn = t.form == kGated ? w.n / 2 : w.n;
      if (bn % kUnit != 0) whole = false;  // the epilogue takes whole groups of columns
      way.blocks[i] = (t.K + kBK - 1) / kBK * (t.form == kJoined ? 2 : 1);
      way.tiles[i] = (t.M + 2 * kRows - 1) / (2 * kRows) * ((t.N + bn - 1) / bn);
      const double units = static_cast<double>(way.tiles[i]) * static_cast<double>(way.blocks[i]);
      flops += units * 2.0 * 2 * kRows * w.n * kBK;
      bytes += units * (2 * kABytes + w.n * kBK * 2);
      if (t.split) {
        way.cut_tiles += way.tiles[i];
        way.cut_work += units * w.block;
        if (way.cut_blocks < way.blocks[i]) way.cut_blocks = way.blocks[i];
      } else {
        way.whole_work += units * w.block + static_cast<double>(way.tiles[i]) * kNextTile;
      }
    }
    if (!whole) continue;
    way.least = flops / 1.8e9;
    if (way.least < bytes / 16e6) way.least = bytes / 16e6;
    ++n_ways;
  }

  // What is added to the longest share: the launch, and with pieces the second launch and their way.
  auto around = [&](const Way& w, int64_t splits) {
    double time = 4.1 + 0.006 * w.width;
    if (splits > 1)
      time += kSumLaunch + kSumPiece * static_cast<double>(splits) +
              static_cast<double>(w.cut_tiles * splits) * (2 * kRows * 4.0 / 5e6) * w.width;
    return time;
  };
  auto room = [&](const Way& w, int64_t splits) {
    return splits == 1 ||
           static_cast<size_t>(w.cut_tiles * splits) * 2 * kRows * static_cast<size_t>(w.width) * 4 <= partial_bytes;
  };
  auto consider = [&](const Way& w, int64_t splits) {
    int64_t first[kMaxProblems + 1] = {};
    double tile_time[kMaxProblems] = {};
    for (int i = 0; i < n; ++i) {
      const bool cut = splits > 1 && tasks[i].split;
      first[i + 1] = first[i] + w.tiles[i] * (cut ? splits : 1);
      tile_time[i] = cut ? static_cast<double>((w.blocks[i] + splits - 1) / splits) * w.block + kCutTile
                         : static_cast<double>(w.blocks[i]) * w.block + kNextTile;
    }
    // The longest share: pair j has the tiles j, j + pairs, ... of all products in turn, and a product
    // gives the pairs from its first tile's on one more than the others. So the longest begins where a
    // product begins.
    double time = w.least;
    for (int i = 0; i < n; ++i) {
      const int64_t j = first[i] % pairs;
      auto before = [&](int64_t end) { return end > j ? (end - j + pairs - 1) / pairs : 0; };
      double share = -kNextTile;
      int64_t done = before(first[0]);
      for (int k = 0; k < n; ++k) {
        const int64_t next = before(first[k + 1]);
        share += static_cast<double>(next - done) * tile_time[k];
        done = next;
      }
      if (time < share) time = share;
    }
    time += around(w, splits);
    if (plan.cost == 0.0 || (splits == 1 ? time <= plan.cost : time < plan.cost)) {
      plan.cost = time;
      plan.width = w.width;
      plan.splits = static_cast<int>(splits);
    }
  };

  for (int i = 0; i < n_ways; ++i) consider(ways[i], 1);
  if (most_splits < 2) return plan;
  // One round of the pairs first: near the best, it rules out most of the other counts by two bounds. A piece's
  // own time falls with their number, so that the counts begin where it fits; the rest only grows with it, and
  // they end where that alone is longer. The choice is the same as without the bounds (enqueueing the gradients of a
  // 64 x 64 weight over 65536 rows took 31 us, gated 40 to 50, and takes 18 to 21 as with few rows).
  for (int i = 0; i < n_ways; ++i) {
    int64_t once = pairs / ways[i].cut_tiles;
    if (once > most_splits) once = most_splits;
    if (once > 1 && room(ways[i], once)) consider(ways[i], once);
  }
  for (int i = 0; i < n_ways; ++i) {
    const Way& w = ways[i];
    const double fits = plan.cost - around(w, 2) + kNextTile - kCutTile;  // for the blocks of one piece
    if (fits <= 0.0) continue;
    int64_t splits = static_cast<int64_t>(static_cast<double>(w.cut_blocks) * w.block / fits);
    if (splits < 2) splits = 2;
    for (; splits <= most_splits && room(w, splits); ++splits) {
      double bound =
          (w.whole_work + w.cut_work + static_cast<double>(w.cut_tiles * splits) * kCutTile) / pairs - kNextTile;
      if (bound < w.least) bound = w.least;
      if (bound + around(w, splits) >= plan.cost) break;
      consider(w, splits);
    }
  }
  return plan;
}

// Room for one piece of 256 x 256 sums on every pair of SMs, where the weights have so few tiles that they
// leave half of the pairs idle and the rows allow two pieces.
size_t weight_partial_bytes(int64_t M, int64_t N, int64_t K, int weights) {
  constexpr int64_t kPairs = 80;
  const int64_t splits = M / (8 * kBK);
  if (N == 0 || K == 0 || splits < 2 || weights == 0) return 0;
  const int64_t tiles_n = (N + kMaxN - 1) / kMaxN, tiles_k = (K + kMaxN - 1) / kMaxN;
  if (tiles_n > kPairs || tiles_k > kPairs || weights * tiles_n * tiles_k > kPairs / 2) return 0;
  const int64_t tiles = weights * tiles_n * tiles_k, most = tiles * splits;
  return static_cast<size_t>(most < kPairs ? most : kPairs) * kMaxN * kMaxN * 4;
}

namespace {

// Whether a tile's sum is longer than an accumulator takes.
bool long_sum(const Task& t, const PairPlan& plan) {
  const int64_t depth = slot_depth(plan.width), blocks = (t.K + depth - 1) / depth;
  const int64_t piece = t.form == kJoined ? 2 * blocks : t.split ? (blocks + plan.splits - 1) / plan.splits : blocks;
  return piece > kMaxPiece / depth;
}

template <int KIND>
cudaError_t run(const Context& c, const Task* tasks, const PairPlan& plan, int n) {
  bool any_long = false;
  for (int i = 0; i < n; ++i) any_long = any_long || long_sum(tasks[i], plan);
  if (tasks[0].form == kGated)
    return any_long ? launch<KIND, true, false, true>(c, tasks, plan, n)
                    : launch<KIND, true, false, false>(c, tasks, plan, n);
  if (any_long) return launch<KIND, false, true, true>(c, tasks, plan, n);
  return plan.splits > 1 ? launch<KIND, false, true, false>(c, tasks, plan, n)
                         : launch<KIND, false, false, false>(c, tasks, plan, n);
}

}  // namespace

cudaError_t run_pair(const Context& c, const Task* tasks, const PairPlan& plan, int n) {
  if (n == 0) return cudaSuccess;
  return c.kind == kBf16 ? run<kBf16>(c, tasks, plan, n) : run<kF16>(c, tasks, plan, n);
}

}  // namespace ff
}  // namespace t2s
