// dropout.cu -- y = drop(x) + r over a matrix.
#include <cuda_runtime.h>

#include <cstdint>

#include "norm_device.cuh"

namespace t2s {
namespace norm {
namespace {

constexpr int kThreads = 256;
constexpr int kAhead = 4;  // words of a thread that are on their way at once

struct DropoutParams {
  DropoutTask t;
  int64_t words, per_row;  // of eight values
  int x_wide, r_wide, y_wide;
};

// INDEX: 32 bits where the words' numbers fit, for the division by a row's words.
template <int KIND, class INDEX>
__global__ void __launch_bounds__(kThreads) dropout_kernel(const __grid_constant__ DropoutParams p) {
  ff::wait_for_earlier_kernels();
  const DropoutTask& t = p.t;
  const uint64_t key = drop_key(t.drop), groups = static_cast<uint64_t>((t.N + 3) / 4);
  const INDEX words = static_cast<INDEX>(p.words), per_row = static_cast<INDEX>(p.per_row);
  const INDEX step = static_cast<INDEX>(gridDim.x) * (kAhead * kThreads);
  for (INDEX first = static_cast<INDEX>(blockIdx.x) * (kAhead * kThreads) + threadIdx.x; first < words; first += step) {
    uint4 x[kAhead], r[kAhead];
    int64_t m[kAhead];
    int n[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const INDEX w = first + i * kThreads;
      m[i] = -1;
      if (w >= words) break;
      const INDEX row = w / per_row;
      m[i] = row;
      n[i] = static_cast<int>(w - row * per_row) * kWord;
      const int left = static_cast<int>(t.N) - n[i];
      x[i] = load_word(t.X.p + m[i] * t.X.ld + n[i], left, p.x_wide);
      if (t.R.p != nullptr) r[i] = load_word(t.R.p + m[i] * t.R.ld + n[i], left, p.r_wide);
    }
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      if (m[i] < 0) break;
      float v[kWord];
      unpack<KIND>(x[i], v);
      drop_word(t.drop, key, static_cast<uint64_t>(m[i]) * groups + static_cast<uint64_t>(n[i] / 4), v);
      if (t.R.p != nullptr) {
        float u[kWord];
        unpack<KIND>(r[i], u);
#pragma unroll
        for (int j = 0; j < kWord; ++j) v[j] += u[j];
      }
      store_word(t.Y.p + m[i] * t.Y.ld + n[i], static_cast<int>(t.N) - n[i], p.y_wide, pack<KIND>(v));
    }
  }
}

template <int KIND>
cudaError_t run(const DropoutTask& t, cudaStream_t stream) {
  DropoutParams p{t};
  p.per_row = (t.N + kWord - 1) / kWord;
  p.words = t.M * p.per_row;
  p.x_wide = wide_rows(t.X.p, t.X.ld, t.M), p.r_wide = wide_rows(t.R.p, t.R.ld, t.M);
  p.y_wide = wide_rows(t.Y.p, t.Y.ld, t.M);
  const int64_t blocks = (p.words + kAhead * kThreads - 1) / (kAhead * kThreads);
  constexpr int64_t kMost = 152 * 4;
  const ff::LaunchShape shape{dim3(static_cast<unsigned>(blocks < kMost ? blocks : kMost)), kThreads, 1, 0};
  return p.words < (int64_t{1} << 31) - kMost * kAhead * kThreads
             ? ff::launch_early(stream, shape, dropout_kernel<KIND, uint32_t>, p)
             : ff::launch_early(stream, shape, dropout_kernel<KIND, uint64_t>, p);
}

}  // namespace

cudaError_t run_dropout(const DropoutTask& t, cudaStream_t stream) {
  return t.kind == ff::kBf16 ? run<ff::kBf16>(t, stream) : run<ff::kF16>(t, stream);
}

}  // namespace norm
}  // namespace t2s
