// ff_elementwise.cu -- the elementwise halves of the feed-forward operators' gradients, and copies of
// operands that the tensor cores' copies cannot read in place.
//
//   linear: dZ = dY * act'(Z), db = sum over rows of dZ
//   gated:  dG = dH * U * act'(G), dU = dH * act(G)
//
// dZ, dG and dU are rounded to the 16-bit type: they are the tensor-core operands of the weight
// and input gradients. db sums the FP32 values before that rounding, in an order that depends on
// the sizes alone. Bound by memory: every value is read or written once, 16 bytes per access
// where rows allow it (4096^2, from HBM: db alone with relu 16.1 us, with gelu 19.1, floor 10.0; both inputs fit
// the L2 cache, and from there it is 9.5 and 14.9, gelu's arithmetic; dG and dU with silu 28 us, floor 25.1).
//
// Inputs are read with plain loads (no __restrict__): these kernels may start before the one that
// writes them has ended (wait_for_earlier_kernels), which read-only loads do not allow for.
#include <cuda_runtime.h>

#include <cstdint>
#include <type_traits>

#include "ff_device.cuh"
#include "ff_internal.h"
#include "ff_math.cuh"
#include "tc_gemm.cuh"

namespace t2s {
namespace ff {
namespace {

constexpr int kThreads = 256;
constexpr int kVec = 8;        // values of a thread in a row: 16 bytes
constexpr int kMaxChunks = 8;  // CTAs that share db's sums: a cluster

struct Source {
  const uint16_t* p;
  int64_t ld;
  int wide;  // rows on 16-byte boundaries
};

// Eight values of a row from column c on as four words, zeros beyond `cols`. Rows that start on odd
// places are read as words with the two ends by themselves, so that nothing outside the row is read.
__device__ __forceinline__ uint4 load8(const Source& s, int64_t r, int64_t c, int64_t cols) {
  const uint16_t* p = s.p + r * s.ld + c;
  if (c + kVec <= cols) {
    if (s.wide) return *reinterpret_cast<const uint4*>(p);
    if ((reinterpret_cast<uintptr_t>(p) & 2u) == 0) {
      const uint32_t* w = reinterpret_cast<const uint32_t*>(p);
      return make_uint4(w[0], w[1], w[2], w[3]);
    }
    const uint32_t* w = reinterpret_cast<const uint32_t*>(p + 1);
    const uint32_t a = p[0], b = w[0], d = w[1], e = w[2], f = p[7];
    return make_uint4(a | b << 16, b >> 16 | d << 16, d >> 16 | e << 16, e >> 16 | f << 16);
  }
  uint32_t v[kVec];
#pragma unroll
  for (int i = 0; i < kVec; ++i) v[i] = c + i < cols ? p[i] : 0u;
  return make_uint4(v[0] | v[1] << 16, v[2] | v[3] << 16, v[4] | v[5] << 16, v[6] | v[7] << 16);
}

constexpr int kPairs = kVec / 2;

template <int KIND>
__device__ __forceinline__ void widen(const uint4& w, uint64_t (&v)[kPairs]) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < kPairs; ++i) {
    const float2 f = to_f32x2<KIND>(u[i]);
    v[i] = pack2(f.x, f.y);
  }
}

template <int KIND>
__device__ __forceinline__ uint4 narrow(const uint64_t (&v)[kPairs]) {
  uint32_t u[4];
#pragma unroll
  for (int i = 0; i < kPairs; ++i) {
    const float2 f = halves(v[i]);
    u[i] = pack_f32<KIND>(f.x, f.y);
  }
  return make_uint4(u[0], u[1], u[2], u[3]);
}

// kGroups threads along a row. Block (x, y): 8 kGroups columns y, y + gridDim.y, ..., the rows of
// chunk x, 256 / kGroups at a time; dZ's rows are 16-byte aligned and padded to whole words. With db the
// chunks are a cluster's CTAs: each leaves its column sums in its shared memory, and the first adds them in
// rank order. With partials each block leaves its column sums there, a row per chunk, for db_sum_kernel.
// Rows and columns are 32-bit (T2S_MAX_DIM is 2^30): with 64-bit ones gelu's slope spills at four blocks to an SM.
template <int KIND, int ACT, int kGroups>
__global__ void __launch_bounds__(kThreads, 4)
    act_backward_kernel(int M, int N, int chunk, Source dy, Source z, uint16_t* dZ, int64_t lddz,
                        uint16_t* db, float* partials) {
  constexpr int kColumns = kGroups * kVec, kLanes = kThreads / kGroups;
  __shared__ float sums[kLanes][kColumns + 1];
  __shared__ float column[kColumns];
  wait_for_earlier_kernels();
  const int group = threadIdx.x % kGroups, row = threadIdx.x / kGroups;
  const int x = static_cast<int>(blockIdx.x), m1 = min((x + 1) * chunk, M);
  for (int c0 = static_cast<int>(blockIdx.y) * kColumns; c0 < N; c0 += static_cast<int>(gridDim.y) * kColumns) {
    const int c = c0 + group * kVec;
    uint64_t sum[kPairs] = {};
    auto take = [&](int m, const uint4& wy, const uint4& wz) {
      uint64_t d[kPairs];
      widen<KIND>(wy, d);
      if constexpr (ACT != T2S_ACT_NONE) {
        uint64_t x[kPairs];
        widen<KIND>(wz, x);
#pragma unroll
        for (int i = 0; i < kPairs; ++i) {
          uint64_t value, slope;
          act_pair_slope<ACT>(x[i], value, slope);
          // The sum takes the unrounded product, whether dZ is stored too or not: left to the compiler,
          // the two could differ in db's last bit.
          sum[i] = fma2(d[i], slope, sum[i]);
          d[i] = mul2(d[i], slope);
        }
      } else {
#pragma unroll
        for (int i = 0; i < kPairs; ++i) sum[i] = add2(sum[i], d[i]);
      }
      if (dZ != nullptr) *reinterpret_cast<uint4*>(dZ + static_cast<int64_t>(m) * lddz + c) = narrow<KIND>(d);
    };
    int m = x * chunk + row;
    if (dy.wide && (ACT == T2S_ACT_NONE || z.wide) && c + kVec <= N) {
      // Two rows' loads before the first row's arithmetic, four blocks to an SM (four rows and three blocks
      // were 16 % slower at 4096^2 with gelu).
      constexpr int kAhead = 2;
      for (; m + (kAhead - 1) * kLanes < m1; m += kAhead * kLanes) {
        uint4 wy[kAhead], wz[kAhead] = {};
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
          wy[j] = *reinterpret_cast<const uint4*>(dy.p + static_cast<int64_t>(m + j * kLanes) * dy.ld + c);
          if (ACT != T2S_ACT_NONE)
            wz[j] = *reinterpret_cast<const uint4*>(z.p + static_cast<int64_t>(m + j * kLanes) * z.ld + c);
        }
#pragma unroll
        for (int j = 0; j < kAhead; ++j) take(m + j * kLanes, wy[j], wz[j]);
      }
    }
    if (c < N)
      for (; m < m1; m += kLanes)
        take(m, load8(dy, m, c, N), ACT != T2S_ACT_NONE ? load8(z, m, c, N) : make_uint4(0, 0, 0, 0));
    if (db == nullptr && partials == nullptr) continue;
#pragma unroll
    for (int i = 0; i < kPairs; ++i) {
      const float2 f = halves(sum[i]);
      sums[row][group * kVec + 2 * i] = f.x;
      sums[row][group * kVec + 2 * i + 1] = f.y;
    }
    __syncthreads();
    if (threadIdx.x < kColumns) {
      float total = 0.0f;
#pragma unroll
      for (int r = 0; r < kLanes; ++r) total += sums[r][threadIdx.x];
      column[threadIdx.x] = total;
      if (partials != nullptr && c0 + static_cast<int>(threadIdx.x) < N)
        partials[static_cast<int64_t>(x) * N + c0 + threadIdx.x] = total;
    }
    if (partials != nullptr) {
      __syncthreads();
      continue;
    }
    cluster_sync_all();
    if (cluster_ctarank() == 0 && threadIdx.x < kColumns && c0 + static_cast<int>(threadIdx.x) < N) {
      // All CTAs' sums on their way before the first is added.
      float part[kMaxChunks], total = 0.0f;
#pragma unroll
      for (int i = 0; i < kMaxChunks; ++i) {
        part[i] = 0.0f;
        if (i < static_cast<int>(gridDim.x))
          asm volatile("ld.shared::cluster.f32 %0, [%1];"
                       : "=f"(part[i])
                       : "r"(tc::map_to_rank(smem_u32(column + threadIdx.x), i)));
      }
#pragma unroll
      for (int i = 0; i < kMaxChunks; ++i) total += part[i];
      db[c0 + threadIdx.x] = from_f32<KIND>(total);
    }
    cluster_sync_all();
  }
}

// 32 columns per block, the partial sums' rows over its warps (65536x64: 1024 rows, db 17.8 us with
// eight warps, 10.1 with 32).
constexpr int kSumWarps = 32;
template <int KIND>
__global__ void __launch_bounds__(32 * kSumWarps) db_sum_kernel(int64_t rows, int64_t N, const float* partials, uint16_t* db) {
  wait_for_earlier_kernels();
  __shared__ float sums[kSumWarps][32];
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  const int64_t n = static_cast<int64_t>(blockIdx.x) * 32 + lane;
  float sum = 0.0f;
  if (n < N) {
#pragma unroll 8
    for (int64_t r = warp; r < rows; r += kSumWarps) sum += partials[r * N + n];
  }
  sums[warp][lane] = sum;
  __syncthreads();
  if (warp != 0 || n >= N) return;
  float total = 0.0f;
#pragma unroll
  for (int w = 0; w < kSumWarps; ++w) total += sums[w][lane];
  db[n] = from_f32<KIND>(total);
}

// i / d of a count of words; a 32-bit division is a fraction of a 64-bit one (copies of 1000x1999 and
// 1999x2001 19.8 -> 17.3 us with the product).
__device__ __forceinline__ int64_t quotient(int64_t i, int64_t d) {
  return (i | d) >> 32 == 0 ? static_cast<int64_t>(static_cast<uint32_t>(i) / static_cast<uint32_t>(d)) : i / d;
}

// One thread per eight values.
template <int KIND, int ACT>
__global__ void __launch_bounds__(kThreads)
    gated_backward_kernel(int64_t M, int64_t N, Source dh, Source g, Source u, uint16_t* dG, uint16_t* dU,
                          int64_t ldd) {
  wait_for_earlier_kernels();
  const int64_t per_row = ldd / kVec, total = M * per_row;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x; i < total;
       i += static_cast<int64_t>(gridDim.x) * kThreads) {
    const int64_t m = quotient(i, per_row), c = (i - m * per_row) * kVec;
    const uint4 wd = load8(dh, m, c, N), wg = load8(g, m, c, N), wu = load8(u, m, c, N);
    uint64_t d[kPairs], x[kPairs], y[kPairs];
    widen<KIND>(wd, d);
    widen<KIND>(wg, x);
    widen<KIND>(wu, y);
#pragma unroll
    for (int j = 0; j < kPairs; ++j) {
      uint64_t value, slope;
      act_pair_slope<ACT>(x[j], value, slope);
      x[j] = mul2(mul2(d[j], y[j]), slope);
      y[j] = mul2(d[j], value);
    }
    *reinterpret_cast<uint4*>(dG + m * ldd + c) = narrow<KIND>(x);
    *reinterpret_cast<uint4*>(dU + m * ldd + c) = narrow<KIND>(y);
  }
}

struct CopyJobs {
  Copy job[kMaxCopies];
  unsigned first[kMaxCopies + 1];  // first block of each
};

// Eight values per thread, written as one word.
__global__ void __launch_bounds__(kThreads) copy_kernel(const __grid_constant__ CopyJobs jobs) {
  wait_for_earlier_kernels();
  int j = 0;
  while (blockIdx.x >= jobs.first[j + 1]) ++j;
  const Copy& c = jobs.job[j];
  const int64_t ldd = (c.cols + kVec - 1) / kVec * kVec, per_row = ldd / kVec, total = c.rows * per_row;
  const int64_t step = static_cast<int64_t>(jobs.first[j + 1] - jobs.first[j]) * kThreads;
  const Source s{c.src, c.ld, 0};
  for (int64_t i = static_cast<int64_t>(blockIdx.x - jobs.first[j]) * kThreads + threadIdx.x; i < total; i += step) {
    const int64_t r = quotient(i, per_row), col = (i - r * per_row) * kVec;
    *reinterpret_cast<uint4*>(c.dst + r * ldd + col) = load8(s, r, col, c.cols);
  }
}

Source source(const uint16_t* p, int64_t ld) { return {p, ld, aligned16(p, ld) ? 1 : 0}; }

template <class F>
cudaError_t for_act(int act, F&& f) {
  switch (act) {
    case T2S_ACT_RELU: return f(std::integral_constant<int, T2S_ACT_RELU>{});
    case T2S_ACT_SILU: return f(std::integral_constant<int, T2S_ACT_SILU>{});
    case T2S_ACT_GELU: return f(std::integral_constant<int, T2S_ACT_GELU>{});
    case T2S_ACT_GELU_TANH: return f(std::integral_constant<int, T2S_ACT_GELU_TANH>{});
    default: return f(std::integral_constant<int, T2S_ACT_NONE>{});
  }
}

unsigned capped(int64_t blocks, int64_t most) { return static_cast<unsigned>(blocks < most ? blocks : most); }

}  // namespace

cudaError_t run_copies(const Context& c, const Copy* copies, int n) {
  if (n == 0) return cudaSuccess;
  CopyJobs jobs = {};
  unsigned blocks = 0;
  for (int i = 0; i < kMaxCopies; ++i) {
    jobs.first[i] = blocks;
    if (i < n) {
      jobs.job[i] = copies[i];
      blocks += capped((copies[i].rows * ((copies[i].cols + kVec - 1) / kVec) + kThreads - 1) / kThreads, 2048);
    }
  }
  jobs.first[kMaxCopies] = blocks;
  return launch_early(c.stream, {dim3(blocks), kThreads, 1, 0}, copy_kernel, jobs);
}

namespace {

// Rows in pieces of 128 bytes where there are blocks enough for the SMs, of 64 bytes otherwise (db of
// 4096^2 with relu is 18 % shorter in pieces of 128, of 1000^2 with gelu a third shorter in pieces of 64).
int groups_of(int64_t N) { return N >= 2048 ? 8 : 4; }

int64_t column_blocks(int64_t N) { return (N + groups_of(N) * kVec - 1) / (groups_of(N) * kVec); }

// Chunks of rows that fill the SMs several times over.
int64_t many_chunks(int64_t M, int64_t N) {
  const int64_t lanes = kThreads / groups_of(N), most = (M + lanes - 1) / lanes;
  int64_t chunks = 2048 / column_blocks(N);
  chunks = chunks < 1 ? 1 : chunks;
  return chunks < most ? chunks : most;
}

// db from partial sums and a second launch where a cluster's eight CTAs per column block are too few to
// keep HBM busy (dZ, db and a 64-wide dX of 16384x1024 54 -> 34 us, 16384x512 31 -> 17, 16384x64 15 -> 8,
// 8192x1024 19 -> 16; but 8192x512 13.4 -> 14.0, 4096x1024 14.3 -> 14.7, 512x1024 8.1 -> 8.5).
bool two_stages(int64_t M, int64_t N) { return M >= 16384 || M * N >= 1 << 23; }

}  // namespace

size_t db_partial_bytes(int64_t M, int64_t N) {
  return N > 0 && two_stages(M, N) ? static_cast<size_t>(many_chunks(M, N)) * static_cast<size_t>(N) * 4 : 0;
}

cudaError_t run_act_backward(const Context& c, int64_t M, int64_t N, int act, const uint16_t* dY,
                             int64_t lddy, const uint16_t* Z, int64_t ldz, uint16_t* dZ,
                             int64_t lddz, uint16_t* db, float* partials) {
  const bool clustered = db != nullptr && !two_stages(M, N);
  const int groups = groups_of(N);
  const int64_t most = (M + kThreads / groups - 1) / (kThreads / groups);
  int64_t chunks = many_chunks(M, N);
  if (clustered)
    for (chunks = kMaxChunks; chunks > most;) chunks /= 2;
  const int64_t chunk = (M + chunks - 1) / chunks;
  const LaunchShape shape{dim3(static_cast<unsigned>(chunks), capped(column_blocks(N), 65535)), kThreads,
                          clustered ? static_cast<int>(chunks) : 1, 0};
  float* parts = db != nullptr && !clustered ? partials : nullptr;
  const cudaError_t e = for_act(act, [&](auto a) {
    constexpr int kAct = decltype(a)::value;
    auto kern = groups == 8
                    ? (c.kind == kBf16 ? act_backward_kernel<kBf16, kAct, 8> : act_backward_kernel<kF16, kAct, 8>)
                    : (c.kind == kBf16 ? act_backward_kernel<kBf16, kAct, 4> : act_backward_kernel<kF16, kAct, 4>);
    return launch_early(c.stream, shape, kern, static_cast<int>(M), static_cast<int>(N), static_cast<int>(chunk),
                        source(dY, lddy), source(Z, ldz), dZ, lddz, clustered ? db : nullptr, parts);
  });
  if (e != cudaSuccess || parts == nullptr) return e;
  return launch_early(c.stream, {dim3(static_cast<unsigned>((N + 31) / 32)), 32 * kSumWarps, 1, 0},
                      c.kind == kBf16 ? db_sum_kernel<kBf16> : db_sum_kernel<kF16>, chunks, N, parts, db);
}

cudaError_t run_gated_backward(const Context& c, int64_t M, int64_t N, int act, const uint16_t* dH,
                               int64_t lddh, const uint16_t* G, int64_t ldg, const uint16_t* U,
                               int64_t ldu, uint16_t* dG, uint16_t* dU, int64_t ldd) {
  const LaunchShape shape{dim3(capped((M * (ldd / kVec) + kThreads - 1) / kThreads, 1 << 20)), kThreads, 1, 0};
  return for_act(act, [&](auto a) {
    constexpr int kAct = decltype(a)::value;
    return launch_early(c.stream, shape,
                        c.kind == kBf16 ? gated_backward_kernel<kBf16, kAct> : gated_backward_kernel<kF16, kAct>, M, N,
                        source(dH, lddh), source(G, ldg), source(U, ldu), dG, dU, ldd);
  });
}

}  // namespace ff
}  // namespace t2s
