// fp8_internal.h -- the 8-bit floating-point operators between their C entry points (fp8_api.cu) and
// the kernels: quantisation, and the product of operands with a scale for each block of 128 of K.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "t2s_internal.h"

namespace t2s {
namespace fp8 {

constexpr int kBlock = 128;  // values of K that share a scale

inline int64_t blocks_of(int64_t n) { return (n + kBlock - 1) / kBlock; }

// Types of quantisation's inputs and of the product's outputs.
enum Wide : int { kF16 = 0, kBf16 = 1, kF32 = 2 };

// Scales: that of row (or group of rows) r and block b lies at p[r * row + b * block].
struct Scales {
  float* p = nullptr;
  int64_t row = 0, block = 0;
};

// Rows of 8-bit values, ld bytes apart, with their scales.
struct Quantized {
  uint8_t* q = nullptr;  // nullptr: not wanted
  int64_t ld = 0;
  Scales s;
};

// X (M x N) in 8 bits along its rows, and along its columns (N rows of M values).
struct QuantizeTask {
  Wide type;
  int64_t M, N;
  const void* X;
  int64_t ldx;
  int format;   // T2S_E4M3 or T2S_E5M2
  bool square;  // a scale for 128 x 128 instead of for 128 values of a row
  Quantized rows, columns;
};
cudaError_t run_quantize(const QuantizeTask& t, cudaStream_t stream);

// C (M x N) = sum over blocks b of K of A_b B_b^T sa[m, b] sb[n / b_group, b].
struct ProductTask {
  Wide type;
  int64_t M, N, K;
  const uint8_t *A, *B;  // M and N rows of K values
  int64_t lda, ldb;
  int format_a, format_b;
  Scales sa, sb;
  int b_group;  // rows of B that share a scale: 1 or 128
  void* C;
  int64_t ldc;
};
cudaError_t run_product(const ProductTask& t, cudaStream_t stream);
// By SM pairs in tiles of 256 rows x `width` (64, 128 or 256) columns (fp8_pair.cu).
struct PairPlan {
  int width = 0;
  double cost = 0.0;  // expected time in microseconds
};
PairPlan plan_pair(const ProductTask& t, int pairs);
cudaError_t run_pair(const ProductTask& t, const PairPlan& plan, cudaStream_t stream, unsigned* status);

// With B's rows along the tensor core's and the sum split over clusters (fp8_rows.cu): rows of A in a tile, CTAs along K,
// and the SMs that their clusters reach.
struct RowsPlan {
  int rows = 0, splits = 1, reach = 0;
  double cost = 0.0;
};
RowsPlan plan_rows(const ProductTask& t, int sms);
cudaError_t run_rows(const ProductTask& t, const RowsPlan& plan, cudaStream_t stream, unsigned* status);

}  // namespace fp8
}  // namespace t2s
