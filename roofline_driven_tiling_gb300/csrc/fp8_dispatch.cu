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
  const int64_t rows = (t.M + 255) / 256;
  const int width = rows * ((t.N + 255) / 256) >= 76 ? 256 : rows * ((t.N + 127) / 128) >= 76 ? 128 : 64;
  return run_pair(t, width, stream, status);
}

}  // namespace fp8
}  // namespace t2s
