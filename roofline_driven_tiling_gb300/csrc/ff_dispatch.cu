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
  int sms = 0;
  cudaError_t e = sm_count(&sms);
  if (e != cudaSuccess) return e;
  Task rest[3];
  int widths[3], left = 0;
  for (int i = 0; i < n; ++i) {
    double pair_cost = 0.0;
    const int width = pair_width(tasks[i], sms / 2, &pair_cost);
    const RowsPlan plan = plan_rows(tasks[i], sms);
    if (plan.cost < pair_cost) {
      if ((e = run_rows(c, tasks[i], plan)) != cudaSuccess) return e;
    } else {
      widths[left] = width;
      rest[left++] = tasks[i];
    }
  }
  return run_pair(c, rest, widths, left);
}

}  // namespace ff
}  // namespace t2s
