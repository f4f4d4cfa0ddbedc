// ff_elementwise.cu -- the elementwise halves of the feed-forward operators' gradients.
//
//   linear: dZ = dY * act'(Z), db = sum over rows of dZ
//   gated:  dG = dH * U * act'(G), dU = dH * act(G)
//
// dZ, dG and dU are rounded to the 16-bit type: they are the tensor-core operands of the weight
// and input gradients. db sums the FP32 values before that rounding.
#include <cuda_runtime.h>

#include <cstdint>
#include <type_traits>

#include "ff_internal.h"
#include "ff_math.cuh"

namespace t2s {
namespace ff {
namespace {

constexpr int kThreads = 256;

// One thread per column, block row y takes the rows of one chunk: partials[y][n].
template <int KIND>
__global__ void __launch_bounds__(kThreads)
    act_backward_kernel(int64_t M, int64_t N, int64_t chunk, int act, const uint16_t* __restrict__ dY,
                        int64_t lddy, const uint16_t* __restrict__ Z, int64_t ldz,
                        uint16_t* __restrict__ dZ, int64_t lddz, float* __restrict__ partials) {
  const int64_t n = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
  if (n >= N) return;
  const int64_t m0 = blockIdx.y * chunk, m1 = m0 + chunk < M ? m0 + chunk : M;
  float sum = 0.0f;
  with_act(act, [&](auto a) {
    for (int64_t m = m0; m < m1; ++m) {
      float value, slope = 1.0f;
      if (decltype(a)::value != T2S_ACT_NONE)
        act_value_slope<decltype(a)::value>(to_f32<KIND>(Z[m * ldz + n]), value, slope);
      const float d = to_f32<KIND>(dY[m * lddy + n]) * slope;
      sum += d;
      if (dZ != nullptr) dZ[m * lddz + n] = from_f32<KIND>(d);
    }
  });
  if (partials != nullptr) partials[static_cast<int64_t>(blockIdx.y) * N + n] = sum;
}

template <int KIND>
__global__ void __launch_bounds__(kThreads)
    db_sum_kernel(int64_t rows, int64_t N, const float* __restrict__ partials, uint16_t* __restrict__ db) {
  const int64_t n = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
  if (n >= N) return;
  float sum = 0.0f;
  for (int64_t r = 0; r < rows; ++r) sum += partials[r * N + n];
  db[n] = from_f32<KIND>(sum);
}

template <int KIND>
__global__ void __launch_bounds__(kThreads)
    gated_backward_kernel(int64_t M, int64_t N, int act, const uint16_t* __restrict__ dH, int64_t lddh,
                          const uint16_t* __restrict__ G, int64_t ldg, const uint16_t* __restrict__ U,
                          int64_t ldu, uint16_t* __restrict__ dG, uint16_t* __restrict__ dU, int64_t ldd) {
  const int64_t n = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
  if (n >= N) return;
  with_act(act, [&](auto a) {
    for (int64_t m = blockIdx.y; m < M; m += gridDim.y) {
      float value, slope;
      act_value_slope<decltype(a)::value>(to_f32<KIND>(G[m * ldg + n]), value, slope);
      const float d = to_f32<KIND>(dH[m * lddh + n]);
      dG[m * ldd + n] = from_f32<KIND>(d * to_f32<KIND>(U[m * ldu + n]) * slope);
      dU[m * ldd + n] = from_f32<KIND>(d * value);
    }
  });
}

// Copies of operands whose rows are not 16-byte aligned: 8 values per thread, written as one word.
__global__ void __launch_bounds__(kThreads) copy_kernel(int64_t rows, int64_t cols, const uint16_t* __restrict__ src,
                                                        int64_t ld, uint16_t* __restrict__ dst, int64_t ldd) {
  const int64_t per_row = ldd / 8, total = rows * per_row;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x; i < total;
       i += static_cast<int64_t>(gridDim.x) * kThreads) {
    const int64_t r = i / per_row, c = (i - r * per_row) * 8;
    uint16_t v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = c + j < cols ? src[r * ld + c + j] : static_cast<uint16_t>(0);
    *reinterpret_cast<uint4*>(dst + r * ldd + c) =
        make_uint4(v[0] | (uint32_t(v[1]) << 16), v[2] | (uint32_t(v[3]) << 16), v[4] | (uint32_t(v[5]) << 16),
                   v[6] | (uint32_t(v[7]) << 16));
  }
}

}  // namespace

cudaError_t run_copy(const Context& c, int64_t rows, int64_t cols, const uint16_t* src, int64_t ld, uint16_t* dst,
                     int64_t ldd) {
  const int64_t blocks = (rows * (ldd / 8) + kThreads - 1) / kThreads;
  copy_kernel<<<static_cast<unsigned>(blocks < 4096 ? blocks : 4096), kThreads, 0, c.stream>>>(rows, cols, src, ld,
                                                                                              dst, ldd);
  return cudaGetLastError();
}

// Chunks of at least 64 rows, at most 128 of them.
int64_t db_partial_rows(int64_t M, int64_t) {
  const int64_t chunks = (M + 63) / 64;
  return chunks < 128 ? chunks : 128;
}

cudaError_t run_act_backward(const Context& c, int64_t M, int64_t N, int act, const uint16_t* dY,
                             int64_t lddy, const uint16_t* Z, int64_t ldz, uint16_t* dZ,
                             int64_t lddz, uint16_t* db, float* partials) {
  const int64_t rows = db_partial_rows(M, N), chunk = (M + rows - 1) / rows;
  const dim3 grid(static_cast<unsigned>((N + kThreads - 1) / kThreads), static_cast<unsigned>(rows));
  float* parts = db != nullptr ? partials : nullptr;
  if (c.kind == kBf16)
    act_backward_kernel<kBf16><<<grid, kThreads, 0, c.stream>>>(M, N, chunk, act, dY, lddy, Z, ldz, dZ, lddz, parts);
  else
    act_backward_kernel<kF16><<<grid, kThreads, 0, c.stream>>>(M, N, chunk, act, dY, lddy, Z, ldz, dZ, lddz, parts);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || db == nullptr) return e;
  if (c.kind == kBf16)
    db_sum_kernel<kBf16><<<grid.x, kThreads, 0, c.stream>>>(rows, N, parts, db);
  else
    db_sum_kernel<kF16><<<grid.x, kThreads, 0, c.stream>>>(rows, N, parts, db);
  return cudaGetLastError();
}

cudaError_t run_gated_backward(const Context& c, int64_t M, int64_t N, int act, const uint16_t* dH,
                               int64_t lddh, const uint16_t* G, int64_t ldg, const uint16_t* U,
                               int64_t ldu, uint16_t* dG, uint16_t* dU, int64_t ldd) {
  const dim3 grid(static_cast<unsigned>((N + kThreads - 1) / kThreads),
                  static_cast<unsigned>(M < 65535 ? M : 65535));
  if (c.kind == kBf16)
    gated_backward_kernel<kBf16><<<grid, kThreads, 0, c.stream>>>(M, N, act, dH, lddh, G, ldg, U, ldu, dG, dU, ldd);
  else
    gated_backward_kernel<kF16><<<grid, kThreads, 0, c.stream>>>(M, N, act, dH, lddh, G, ldg, U, ldu, dG, dU, ldd);
  return cudaGetLastError();
}

}  // namespace ff
}  // namespace t2s
