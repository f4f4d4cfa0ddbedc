// fp8_dispatch.cu -- which kernel takes a product of 8-bit operands: the one whose own estimate of the time (plan_pair,
// plan_rows) is shorter.
#include <cuda_runtime.h>

#include <cstdint>

#include "fp8_internal.h"

namespace t2s {
namespace fp8 {

cudaError_t run_product(const ProductTask& given, cudaStream_t stream) {
  constexpr int kSms = 152;
  ProductTask t = given;
  // The stride of a single row is never used, but encoded: one that keeps 16-byte boundaries.
  if (t.M == 1) t.lda = (t.K + 15) / 16 * 16;
  if (t.N == 1) t.ldb = (t.K + 15) / 16 * 16;
  unsigned* status = nullptr;
  cudaError_t e = device_status_word(&status);
  if (e != cudaSuccess) return e;
  const PairPlan pair = plan_pair(t, kSms / 2);
  const RowsPlan rows = plan_rows(t, kSms);
  return rows.cost < pair.cost ? run_rows(t, rows, stream, status) : run_pair(t, pair, stream, status);
}

}  // namespace fp8
}  // namespace t2s
