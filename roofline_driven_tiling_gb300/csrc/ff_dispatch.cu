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
  int widths[kMaxProblems], own_widths[kMaxProblems], rows = 0, pairs = 0;
  double all_pair = kStart, mixed = 0.0;
  for (int i = 0; i < n; ++i) {
    double cost = 0.0;
    widths[i] = pair_width(tasks[i], sms / 2, &cost);
    all_pair += cost - kStart;
    const double alone = plan_rows(&tasks[i], 1, sms).cost;
    mixed += (alone < cost ? alone : cost) - kStart;
    if (alone < cost) {
      by_rows[rows++] = tasks[i];
    } else {
      own_widths[pairs] = widths[i];
      by_pair[pairs++] = tasks[i];
    }
  }
  mixed += kStart + (rows > 0 && pairs > 0 ? kLaunch : 0.0);
  const RowsPlan plan = plan_rows(tasks, n, sms);
  if (plan.cost < all_pair && plan.cost < mixed) return run_rows(c, tasks, plan, n);
  if (all_pair <= mixed) return run_pair(c, tasks, widths, n);
  if (rows > 0 && (e = run_rows(c, by_rows, plan_rows(by_rows, rows, sms), rows)) != cudaSuccess) return e;
  return run_pair(c, by_pair, own_widths, pairs);
}

}  // namespace ff
}  // namespace t2s
