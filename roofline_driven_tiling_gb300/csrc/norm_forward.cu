// norm_forward.cu -- r = scale x + gate drop(post(h)), y = norm(r).
#include <cuda_runtime.h>

#include <cstdint>

#include "norm_device.cuh"

namespace t2s {
namespace norm {
namespace {

constexpr int kWideThreads = 1024;

// Rows of any length: a block per row, passes over memory. Every value of r is written and read by the same
// thread.
template <int KIND>
__global__ void __launch_bounds__(kWideThreads) wide_forward_kernel(const __grid_constant__ ForwardTask t) {
  __shared__ float room[64];
  ff::wait_for_earlier_kernels();
  const int64_t groups = (t.N + 3) / 4, rows_per_gate = t.M / t.gates;
  const float inv_n = 1.0f / static_cast<float>(t.N);
  const uint64_t key = t.drop.dropped != 0 ? drop_key(t.drop) : 0;
  for (int64_t m = blockIdx.x; m < t.M; m += gridDim.x) {
    const uint16_t* x = t.X.p + m * t.X.ld;
    const uint16_t* r = x;
    if (t.H.p != nullptr) {
      const uint16_t* h = t.H.p + m * t.H.ld;
      float s[1] = {0.0f}, mean = 0.0f, rstd = 1.0f;
      if (t.post == T2S_NORM_LAYER) {
        for (int64_t n = threadIdx.x; n < t.N; n += kWideThreads) s[0] += ff::to_f32<KIND>(h[n]);
        block_sums(s, room);
        mean = s[0] * inv_n;
      }
      if (t.post != T2S_NORM_NONE) {
        s[0] = 0.0f;
        for (int64_t n = threadIdx.x; n < t.N; n += kWideThreads) {
          const float c = ff::to_f32<KIND>(h[n]) - mean;
          s[0] = fmaf(c, c, s[0]);
        }
        block_sums(s, room);
        rstd = rsqrtf(s[0] * inv_n + t.eps);
      }
      uint16_t* out = t.R.p + m * t.R.ld;
      const uint16_t* gate = t.gate.p == nullptr ? nullptr : t.gate.p + m / rows_per_gate * t.gate.ld;
      for (int64_t n = threadIdx.x; n < t.N; n += kWideThreads) {
        float v = ff::to_f32<KIND>(h[n]);
        if (t.post != T2S_NORM_NONE)
          v = fmaf((v - mean) * rstd, at<KIND>(t.post_weight, n, 1.0f), at<KIND>(t.post_bias, n, 0.0f));
        if (t.drop.dropped != 0)
          v = drop(v, drop_bits(key, static_cast<uint64_t>(m * groups + n / 4)), n & 3, t.drop.dropped, t.drop.factor);
        out[n] = ff::from_f32<KIND>(fmaf(at<KIND>(gate, n, 1.0f), v, t.scale * ff::to_f32<KIND>(x[n])));
      }
      r = out;
    }
    if (t.norm == T2S_NORM_NONE) continue;
    float s[1] = {0.0f}, mean = 0.0f;
    if (t.norm == T2S_NORM_LAYER) {
      for (int64_t n = threadIdx.x; n < t.N; n += kWideThreads) s[0] += ff::to_f32<KIND>(r[n]);
      block_sums(s, room);
      mean = s[0] * inv_n;
      s[0] = 0.0f;
    }
    for (int64_t n = threadIdx.x; n < t.N; n += kWideThreads) {
      const float c = ff::to_f32<KIND>(r[n]) - mean;
      s[0] = fmaf(c, c, s[0]);
    }
    block_sums(s, room);
    const float rstd = rsqrtf(s[0] * inv_n + t.eps);
    uint16_t* y = t.Y.p + m * t.Y.ld;
    for (int64_t n = threadIdx.x; n < t.N; n += kWideThreads)
      y[n] = ff::from_f32<KIND>(
          fmaf((ff::to_f32<KIND>(r[n]) - mean) * rstd, at<KIND>(t.weight, n, 1.0f), at<KIND>(t.bias, n, 0.0f)));
  }
}

template <int KIND>
cudaError_t run(const ForwardTask& t, cudaStream_t stream) {
  const unsigned blocks = static_cast<unsigned>(t.M < 304 ? t.M : 304);
  return ff::launch_early(stream, {dim3(blocks), kWideThreads, 1, 0}, wide_forward_kernel<KIND>, t);
}

}  // namespace

cudaError_t run_forward(const ForwardTask& t, cudaStream_t stream) {
  return t.kind == ff::kBf16 ? run<ff::kBf16>(t, stream) : run<ff::kF16>(t, stream);
}

}  // namespace norm
}  // namespace t2s
