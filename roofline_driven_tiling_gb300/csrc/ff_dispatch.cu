// ff_dispatch.cu -- which kernel takes a product of the feed-forward operators: the one whose own
// estimate of the time (plan_rows, plan_pair) is shorter.
#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>

#include "ff_internal.h"

namespace t2s {
namespace ff {
namespace {

// Multiprocessors of the current device, looked up once per device.
cudaError_t sm_count(int* out) {
  constexpr int kMaxDevices = 64;
  static std::atomic<int> known[kMaxDevices];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
  int n = known[dev].load(std::memory_order_relaxed);
  if (n == 0) {
    if ((e = cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess) return e;
    known[dev].store(n, std::memory_order_relaxed);
  }
  *out = n;
  return cudaSuccess;
}

}  // namespace

cudaError_t run_products(const Context& c, const Task* tasks, int n) {
  if (n == 0) return cudaSuccess;
  int sms = 0;
  cudaError_t e = sm_count(&sms);
  if (e != cudaSuccess) return e;
  // All by one kernel, in one launch, or each by the one that is quicker for it alone.
  constexpr double kStart = 4.0, kLaunch = 2.0;  // of a lone launch; of one more
  Task by_rows[kMaxProblems], by_pair[kMaxProblems];
  int rows = 0, pairs = 0;
  if (n > 1) {
    for (int i = 0; i < n; ++i) {
      if (plan_rows(&tasks[i], 1, sms).cost < plan_pair(&tasks[i], 1, sms / 2, c.partial_bytes).cost) {
        by_rows[rows++] = tasks[i];
      } else {
        by_pair[pairs++] = tasks[i];
      }
    }
  }
  const PairPlan all_pair = plan_pair(tasks, n, sms / 2, c.partial_bytes);
  const RowsPlan all_rows = plan_rows(tasks, n, sms);
  if (rows > 0 && pairs > 0) {
    const PairPlan some_pair = plan_pair(by_pair, pairs, sms / 2, c.partial_bytes);
    const RowsPlan some_rows = plan_rows(by_rows, rows, sms);
    const double mixed = some_pair.cost + some_rows.cost - kStart + kLaunch;
    if (mixed < all_pair.cost && mixed < all_rows.cost) {
      if ((e = run_rows(c, by_rows, some_rows, rows)) != cudaSuccess) return e;
      return run_pair(c, by_pair, some_pair, pairs);
    }
  }
  return all_rows.cost < all_pair.cost ? run_rows(c, tasks, all_rows, n) : run_pair(c, tasks, all_pair, n);
}

}  // namespace ff
}  // namespace t2s
