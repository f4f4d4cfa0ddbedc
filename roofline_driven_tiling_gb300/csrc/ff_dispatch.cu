// ff_dispatch.cu -- which kernel takes a product of the feed-forward operators: the one whose own
// estimate of the time (plan_rows, pair_width) is shorter.
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
      double cost = 0.0;
      pair_width(&tasks[i], 1, sms / 2, &cost);
      if (plan_rows(&tasks[i], 1, sms).cost < cost) {
        by_rows[rows++] = tasks[i];
      } else {
        by_pair[pairs++] = tasks[i];
      }
    }
  }
  double all_pair = 0.0;
  const int width = pair_width(tasks, n, sms / 2, &all_pair);
  const RowsPlan plan = plan_rows(tasks, n, sms);
  if (rows > 0 && pairs > 0) {
    double some_pair = 0.0;
    const int some_width = pair_width(by_pair, pairs, sms / 2, &some_pair);
    const RowsPlan some_rows = plan_rows(by_rows, rows, sms);
    const double mixed = some_pair + some_rows.cost - kStart + kLaunch;
    if (mixed < all_pair && mixed < plan.cost) {
      if ((e = run_rows(c, by_rows, some_rows, rows)) != cudaSuccess) return e;
      return run_pair(c, by_pair, some_width, pairs);
    }
  }
  return plan.cost < all_pair ? run_rows(c, tasks, plan, n) : run_pair(c, tasks, width, n);
}

}  // namespace ff
}  // namespace t2s
