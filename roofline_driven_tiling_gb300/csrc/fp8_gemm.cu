// fp8_gemm.cu -- the product of 8-bit operands with a scale for each block of 128 of K, in FP32 on the CUDA
// cores: 64 x 64 outputs per CTA, the sum of a block of K first, then its scales.
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "ff_device.cuh"
#include "ff_math.cuh"
#include "fp8_internal.h"

namespace t2s {
namespace fp8 {
namespace {

constexpr int kTile = 64, kDepth = 32;

__device__ __forceinline__ float value_of(uint8_t v, int format) {
  return __half2float(__half(__nv_cvt_fp8_to_halfraw(v, format == T2S_E4M3 ? __NV_E4M3 : __NV_E5M2)));
}

__global__ void __launch_bounds__(256) product_kernel(const __grid_constant__ ProductTask t, int64_t tiles_n) {
  __shared__ float a[kDepth][kTile + 1], b[kDepth][kTile + 1];
  ff::wait_for_earlier_kernels();
  const int64_t m0 = blockIdx.x / tiles_n * kTile, n0 = blockIdx.x % tiles_n * kTile;
  const int ty = threadIdx.x / 16, tx = threadIdx.x % 16;
  float sum[4][4] = {};
  for (int64_t k0 = 0; k0 < t.K; k0 += kBlock) {
    float part[4][4] = {};
    for (int64_t k1 = k0; k1 < k0 + kBlock && k1 < t.K; k1 += kDepth) {
      __syncthreads();
      for (int i = threadIdx.x; i < kTile * kDepth; i += 256) {
        const int r = i / kDepth, k = i % kDepth;
        a[k][r] = m0 + r < t.M && k1 + k < t.K ? value_of(t.A[(m0 + r) * t.lda + k1 + k], t.format_a) : 0.0f;
        b[k][r] = n0 + r < t.N && k1 + k < t.K ? value_of(t.B[(n0 + r) * t.ldb + k1 + k], t.format_b) : 0.0f;
      }
      __syncthreads();
      for (int k = 0; k < kDepth; ++k)
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) part[i][j] = fmaf(a[k][ty + 16 * i], b[k][tx + 16 * j], part[i][j]);
    }
    const int64_t kb = k0 / kBlock;
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int64_t m = m0 + ty + 16 * i, n = n0 + tx + 16 * j;
        if (m < t.M && n < t.N)
          sum[i][j] = fmaf(part[i][j], t.sa.p[m * t.sa.row + kb * t.sa.block] *
                                           t.sb.p[n / t.b_group * t.sb.row + kb * t.sb.block], sum[i][j]);
      }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int64_t m = m0 + ty + 16 * i, n = n0 + tx + 16 * j;
      if (m >= t.M || n >= t.N) continue;
      const int64_t at = m * t.ldc + n;
      if (t.type == kF32) {
        static_cast<float*>(t.C)[at] = sum[i][j];
      } else {
        static_cast<uint16_t*>(t.C)[at] =
            t.type == kBf16 ? ff::from_f32<ff::kBf16>(sum[i][j]) : ff::from_f32<ff::kF16>(sum[i][j]);
      }
    }
}

}  // namespace

cudaError_t run_product(const ProductTask& t, cudaStream_t stream) {
  const int64_t tiles_m = (t.M + kTile - 1) / kTile, tiles_n = (t.N + kTile - 1) / kTile;
  if (tiles_m > 0x7fffffff / tiles_n) return cudaErrorInvalidConfiguration;
  return ff::launch_early(stream, {dim3(static_cast<unsigned>(tiles_m * tiles_n)), 256, 1, 0}, product_kernel, t, tiles_n);
}

}  // namespace fp8
}  // namespace t2s
