// fp8_dispatch.cu -- which kernel takes a product of 8-bit operands.
#include <cuda_runtime.h>

#include <cstdint>

#include "fp8_internal.h"

namespace t2s {
namespace fp8 {

cudaError_t run_product(const ProductTask& given, cudaStream_t stream) {
  ProductTask t = given;
  // The stride of a single row is never used, but encoded: one that keeps 16-byte boundaries.
  if (t.M == 1) t.lda = (t.K + 15) / 16 * 16;
  if (t.N == 1) t.ldb = (t.K + 15) / 16 * 16;
  unsigned* status = nullptr;
  cudaError_t e = device_status_word(&status);
  if (e != cudaSuccess) return e;
  // The tile width with the shortest rounds of all pairs of SMs: a block of 128 of K takes a pair 0.28, 0.32 or 0.5 us in tiles
  // of 64, 128 or 256 columns (with a scale for every column 0.30, 0.58, 0.9), and a tile's end 1.5 us.
  constexpr int64_t kPairs = 76;
  static constexpr int kWidths[] = {256, 128, 64};
  static constexpr double kBlockTime[2][3] = {{0.5, 0.32, 0.28}, {0.9, 0.58, 0.30}};
  int width = 0;
  double best = 0.0;
  for (int i = 0; i < 3; ++i) {
    const int64_t tiles = (t.M + 255) / 256 * ((t.N + kWidths[i] - 1) / kWidths[i]);
    const double time = static_cast<double>((tiles + kPairs - 1) / kPairs) *
                        (static_cast<double>(blocks_of(t.K)) * kBlockTime[t.b_group == 1][i] + 1.5);
    if (width == 0 || time < best) {
      width = kWidths[i];
      best = time;
    }
  }
  return run_pair(t, width, stream, status);
}

}  // namespace fp8
}  // namespace t2s
