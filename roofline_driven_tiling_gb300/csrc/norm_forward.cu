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

// Rows of up to kMostWords words a thread and 1024 threads: a group of threads keeps a row in registers, C words of
// eight values a thread, the next row's words on their way meanwhile.
struct RowParams {
  ForwardTask t;
  int threads;  // of a row
  int x_wide, h_wide, r_wide, y_wide, gate_wide, vectors_wide;
};

template <int KIND, int C, int THREADS>
__global__ void __launch_bounds__(THREADS) row_forward_kernel(const __grid_constant__ RowParams p) {
  __shared__ float rooms[Group::kRoomFloats];
  ff::wait_for_earlier_kernels();
  const ForwardTask& t = p.t;
  Group group(p.threads, rooms);
  const int n = static_cast<int>(t.N);
  const int64_t step = static_cast<int64_t>(gridDim.x) * (blockDim.x / p.threads);
  const int64_t groups = (t.N + 3) / 4, rows_per_gate = t.M / t.gates;
  const float inv_n = 1.0f / static_cast<float>(n);
  const uint64_t key = t.drop.dropped != 0 ? drop_key(t.drop) : 0;
  const bool has_h = t.H.p != nullptr;
  int64_t m = static_cast<int64_t>(blockIdx.x) * (blockDim.x / p.threads) + group.index;
  uint4 x[C], h[C];
  auto fetch = [&](int64_t row) {
    if (row >= t.M) return;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int at = (group.rank + c * p.threads) * kWord;
      x[c] = h[c] = make_uint4(0, 0, 0, 0);
      if (at >= n) continue;
      x[c] = load_word(t.X.p + row * t.X.ld + at, n - at, p.x_wide);
      if (has_h) h[c] = load_word(t.H.p + row * t.H.ld + at, n - at, p.h_wide);
    }
  };
  fetch(m);
  for (; m < t.M; m += step) {
    float v[C][kWord];
    uint4 r[C];
    // Values beyond the row's end are 0 and stay 0 in the sums.
    auto centred = [&](int kind, float& rstd) {
      float s[1] = {0.0f};
      if (kind == T2S_NORM_LAYER) {
#pragma unroll
        for (int c = 0; c < C; ++c)
#pragma unroll
          for (int i = 0; i < kWord; ++i) s[0] += v[c][i];
        group.sums(s);
        const float mean = s[0] * inv_n;
#pragma unroll
        for (int c = 0; c < C; ++c)
#pragma unroll
          for (int i = 0; i < kWord; ++i)
            if ((group.rank + c * p.threads) * kWord + i < n) v[c][i] -= mean;
        s[0] = 0.0f;
      }
#pragma unroll
      for (int c = 0; c < C; ++c)
#pragma unroll
        for (int i = 0; i < kWord; ++i) s[0] = fmaf(v[c][i], v[c][i], s[0]);
      group.sums(s);
      rstd = rsqrtf(s[0] * inv_n + t.eps);
    };
    if (has_h) {
#pragma unroll
      for (int c = 0; c < C; ++c) unpack<KIND>(h[c], v[c]);
#pragma unroll
      for (int c = 0; c < C; ++c) r[c] = x[c];
      fetch(m + step);
      float rstd = 1.0f;
      if (t.post != T2S_NORM_NONE) centred(t.post, rstd);
      const uint16_t* gate = t.gate.p == nullptr ? nullptr : t.gate.p + (t.gates == 1 ? 0 : m / rows_per_gate * t.gate.ld);
#pragma unroll
      for (int c = 0; c < C; ++c) {
        const int at = (group.rank + c * p.threads) * kWord, left = n - at;
        if (left <= 0) continue;
        float w[kWord], b[kWord];
        if (t.post != T2S_NORM_NONE) {
          parameter<KIND>(t.post_weight, at, left, p.vectors_wide, 1.0f, w);
          parameter<KIND>(t.post_bias, at, left, p.vectors_wide, 0.0f, b);
#pragma unroll
          for (int i = 0; i < kWord; ++i) v[c][i] = fmaf(v[c][i] * rstd, w[i], b[i]);
        }
        if (t.drop.dropped != 0) drop_word(t.drop, key, static_cast<uint64_t>(m * groups + at / 4), v[c]);
        parameter<KIND>(gate, at, left, p.gate_wide, 1.0f, w);
        unpack<KIND>(r[c], b);
#pragma unroll
        for (int i = 0; i < kWord; ++i) v[c][i] = fmaf(w[i], v[c][i], t.scale * b[i]);
        r[c] = pack<KIND>(v[c]);
        store_word(t.R.p + m * t.R.ld + at, left, p.r_wide, r[c]);
        unpack<KIND>(r[c], v[c]);
#pragma unroll
        for (int i = 0; i < kWord; ++i)
          if (i >= left) v[c][i] = 0.0f;
      }
    } else {
#pragma unroll
      for (int c = 0; c < C; ++c) unpack<KIND>(x[c], v[c]);
      fetch(m + step);
    }
    if (t.norm == T2S_NORM_NONE) continue;
    float rstd;
    centred(t.norm, rstd);
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int at = (group.rank + c * p.threads) * kWord, left = n - at;
      if (left <= 0) continue;
      float w[kWord], b[kWord];
      parameter<KIND>(t.weight, at, left, p.vectors_wide, 1.0f, w);
      parameter<KIND>(t.bias, at, left, p.vectors_wide, 0.0f, b);
#pragma unroll
      for (int i = 0; i < kWord; ++i) v[c][i] = fmaf(v[c][i] * rstd, w[i], b[i]);
      store_word(t.Y.p + m * t.Y.ld + at, left, p.y_wide, pack<KIND>(v[c]));
    }
  }
}

constexpr int kSms = 152;

template <int KIND, int C, int THREADS>
cudaError_t run_rows(const ForwardTask& t, int threads, cudaStream_t stream) {
  RowParams p{t, threads};
  p.x_wide = wide_rows(t.X.p, t.X.ld, t.M), p.h_wide = wide_rows(t.H.p, t.H.ld, t.M);
  p.r_wide = wide_rows(t.R.p, t.R.ld, t.M), p.y_wide = wide_rows(t.Y.p, t.Y.ld, t.M);
  p.gate_wide = wide_rows(t.gate.p, t.gate.ld, t.gates);
  p.vectors_wide = wide_rows(t.weight, 0, 1) && wide_rows(t.bias, 0, 1) && wide_rows(t.post_weight, 0, 1) &&
                   wide_rows(t.post_bias, 0, 1);
  const int rows = THREADS / threads;
  const int64_t blocks = (t.M + rows - 1) / rows, most = kSms * (1536 / THREADS > 0 ? 1536 / THREADS : 1);
  return ff::launch_early(stream, {dim3(static_cast<unsigned>(blocks < most ? blocks : most)), rows * threads, 1, 0},
                          row_forward_kernel<KIND, C, THREADS>, p);
}

// A row of up to 1024 values by one warp (no barriers), up to 8192 in two words a thread, up to 16384 with as many
// threads as a block has; longer ones in passes over memory.
template <int KIND>
cudaError_t run(const ForwardTask& t, cudaStream_t stream) {
  const int64_t words = (t.N + kWord - 1) / kWord;
  if (words <= 32) return run_rows<KIND, 1, 256>(t, 32, stream);
  if (words <= 64) return run_rows<KIND, 2, 256>(t, 32, stream);
  if (words <= 128) return run_rows<KIND, 4, 256>(t, 32, stream);
  const int threads = static_cast<int>((words + 63) / 64 * 32);
  if (threads <= 256) return run_rows<KIND, 2, 256>(t, threads, stream);
  if (threads <= 512) return run_rows<KIND, 2, 512>(t, threads, stream);
  if (threads <= 1024) return run_rows<KIND, 2, 1024>(t, threads, stream);
  const unsigned blocks = static_cast<unsigned>(t.M < 2 * kSms ? t.M : 2 * kSms);
  return ff::launch_early(stream, {dim3(blocks), kWideThreads, 1, 0}, wide_forward_kernel<KIND>, t);
}

}  // namespace

cudaError_t run_forward(const ForwardTask& t, cudaStream_t stream) {
  return t.kind == ff::kBf16 ? run<ff::kBf16>(t, stream) : run<ff::kF16>(t, stream);
}

}  // namespace norm
}  // namespace t2s
