// dropout.cu -- y = drop(x) + r over a matrix.
#include <cuda_runtime.h>

#include <cstdint>

#include "norm_device.cuh"

namespace t2s {
namespace norm {
namespace {

constexpr int kThreads = 256;

// A thread takes the four values of one output of the generator.
template <int KIND>
__global__ void __launch_bounds__(kThreads) dropout_kernel(const __grid_constant__ DropoutTask t, int64_t groups) {
  ff::wait_for_earlier_kernels();
  const uint64_t key = drop_key(t.drop);
  const int64_t all = t.M * groups, step = static_cast<int64_t>(gridDim.x) * kThreads;
  for (int64_t g = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x; g < all; g += step) {
    const int64_t m = g / groups, n = (g - m * groups) * 4;
    const uint64_t bits = drop_bits(key, static_cast<uint64_t>(g));
    for (int j = 0; j < 4 && n + j < t.N; ++j) {
      const float v = drop(ff::to_f32<KIND>(t.X.p[m * t.X.ld + n + j]), bits, j, t.drop.dropped, t.drop.factor);
      t.Y.p[m * t.Y.ld + n + j] =
          ff::from_f32<KIND>(t.R.p == nullptr ? v : v + ff::to_f32<KIND>(t.R.p[m * t.R.ld + n + j]));
    }
  }
}

template <int KIND>
cudaError_t run(const DropoutTask& t, cudaStream_t stream) {
  const int64_t groups = (t.N + 3) / 4, blocks = (t.M * groups + kThreads - 1) / kThreads;
  const unsigned grid = static_cast<unsigned>(blocks < 152 * 8 ? blocks : 152 * 8);
  return ff::launch_early(stream, {dim3(grid), kThreads, 1, 0}, dropout_kernel<KIND>, t, groups);
}

}  // namespace

cudaError_t run_dropout(const DropoutTask& t, cudaStream_t stream) {
  return t.kind == ff::kBf16 ? run<ff::kBf16>(t, stream) : run<ff::kF16>(t, stream);
}

}  // namespace norm
}  // namespace t2s
