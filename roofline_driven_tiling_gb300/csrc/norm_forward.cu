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

// Rows of up to 16384 values: a group of threads keeps a row in registers, C words of eight values a thread, the next
// row's words on their way meanwhile. A thread's words of the parameters lie in shared memory, at places of its own.
struct RowParams {
  row::View x, h, r, y, vector[5];  // see Vector
  int slot[5];                      // of a vector's words in shared memory; -1: absent, or a gate that changes
  int64_t M, rows_per_gate;
  int N, threads;  // threads of a row
  int norm, post;
  float scale, eps;
  Dropout drop;
};
enum Vector : int { kPostWeight = 0, kPostBias = 1, kGate = 2, kWeight = 3, kBias = 4 };

// Blocks that an SM holds: 64 registers a thread, four words a thread twice as many.
template <int C, int THREADS>
constexpr int blocks_of() {
  return (C == 4 ? 512 : 1024) / THREADS;
}

template <int KIND, bool WIDE, int C, int THREADS>
__global__ void __launch_bounds__(THREADS, blocks_of<C, THREADS>()) row_forward_kernel(const __grid_constant__ RowParams p) {
  extern __shared__ uint4 words[];
  __shared__ float rooms[row::Group::kRoomFloats];
  ff::wait_for_earlier_kernels();
  row::Group group(p.threads, rooms);
  const int n = p.N, rows_at_once = static_cast<int>(blockDim.x) / p.threads;
  const int64_t step = static_cast<int64_t>(gridDim.x) * rows_at_once;
  const uint64_t groups = static_cast<uint64_t>((static_cast<int64_t>(n) + 3) / 4);
  const float inv_n = 1.0f / static_cast<float>(n);
  const uint64_t key = p.drop.dropped != 0 ? drop_key(p.drop) : 0;
  const bool has_h = p.h.p != nullptr;
  auto column = [&](int c) { return (group.rank + c * p.threads) * row::kWord; };
  auto parameter = [&](int vector, int c) -> uint4& {
    return words[(p.slot[vector] * C + c) * static_cast<int>(blockDim.x) + static_cast<int>(threadIdx.x)];
  };
#pragma unroll
  for (int i = 0; i < 5; ++i)
    if (p.slot[i] >= 0)
#pragma unroll
      for (int c = 0; c < C; ++c) parameter(i, c) = row::load_word<WIDE>(p.vector[i], p.vector[i].p + column(c), n - column(c));

  uint4 x[C], h[C];
  auto fetch = [&](int64_t m) {
    if (m >= p.M) return;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      x[c] = row::load_word<WIDE>(p.x, p.x.p + m * p.x.ld + column(c), n - column(c));
      if (has_h) h[c] = row::load_word<WIDE>(p.h, p.h.p + m * p.h.ld + column(c), n - column(c));
    }
  };
  uint64_t v[C][4];
  // The mean off the values (layer), and 1 / the root of their mean square.
  auto scale_of = [&](int kind) {
    float s[1] = {0.0f};
    if (kind == T2S_NORM_LAYER) {
#pragma unroll
      for (int c = 0; c < C; ++c) s[0] += row::sum(v[c]);
      group.sums(s);
      const uint64_t mean = row::both(-s[0] * inv_n);
#pragma unroll
      for (int c = 0; c < C; ++c) {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[c][i] = row::add2(v[c][i], mean);
        row::clear_from<WIDE>(v[c], n - column(c));
      }
      s[0] = 0.0f;
    }
#pragma unroll
    for (int c = 0; c < C; ++c) s[0] += row::dot(v[c], v[c]);
    group.sums(s);
    return rsqrtf(s[0] * inv_n + p.eps);
  };
  // A norm's weight and bias on the values times `rstd`.
  auto affine = [&](float rstd, int weight, int bias, int c) {
    uint64_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) v[c][i] = row::mul2(v[c][i], row::both(rstd));
    if (p.slot[weight] >= 0) {
      row::unpack<KIND>(parameter(weight, c), w);
#pragma unroll
      for (int i = 0; i < 4; ++i) v[c][i] = row::mul2(v[c][i], w[i]);
    }
    if (p.slot[bias] >= 0) {
      row::unpack<KIND>(parameter(bias, c), w);
#pragma unroll
      for (int i = 0; i < 4; ++i) v[c][i] = row::add2(v[c][i], w[i]);
    }
  };

  int64_t m = static_cast<int64_t>(blockIdx.x) * rows_at_once + group.index;
  fetch(m);
  for (; m < p.M; m += step) {
    if (has_h) {
      uint4 r[C];
#pragma unroll
      for (int c = 0; c < C; ++c) {
        row::unpack<KIND>(h[c], v[c]);
        r[c] = x[c];
      }
      fetch(m + step);
      const float rstd = p.post != T2S_NORM_NONE ? scale_of(p.post) : 1.0f;
#pragma unroll
      for (int c = 0; c < C; ++c) {
        const int at = column(c);
        uint64_t u[4];
        if (p.post != T2S_NORM_NONE) affine(rstd, kPostWeight, kPostBias, c);
        if (p.drop.dropped != 0) {
          row::Keep keep;
          keep.draw(key, static_cast<uint64_t>(m) * groups + static_cast<uint64_t>(at / 4), p.drop.dropped);
          keep.apply(v[c], p.drop.factor);
        }
        if (p.vector[kGate].p != nullptr) {
          row::unpack<KIND>(p.slot[kGate] >= 0
                                ? parameter(kGate, c)
                                : row::load_word<WIDE>(p.vector[kGate], p.vector[kGate].p + m / p.rows_per_gate * p.vector[kGate].ld + at, n - at),
                            u);
#pragma unroll
          for (int i = 0; i < 4; ++i) v[c][i] = row::mul2(v[c][i], u[i]);
        }
        row::unpack<KIND>(r[c], u);
#pragma unroll
        for (int i = 0; i < 4; ++i) v[c][i] = row::fma2(u[i], row::both(p.scale), v[c][i]);
        // The norm that follows is of the rounded values.
        r[c] = row::pack<KIND>(v[c]);
        row::store_word<WIDE>(p.r, p.r.p + m * p.r.ld + at, n - at, r[c]);
        row::unpack<KIND>(r[c], v[c]);
        row::clear_from<WIDE>(v[c], n - at);
      }
    } else {
#pragma unroll
      for (int c = 0; c < C; ++c) row::unpack<KIND>(x[c], v[c]);
      fetch(m + step);
    }
    if (p.norm == T2S_NORM_NONE) continue;
    const float rstd = scale_of(p.norm);
#pragma unroll
    for (int c = 0; c < C; ++c) {
      affine(rstd, kWeight, kBias, c);
      row::store_word<WIDE>(p.y, p.y.p + m * p.y.ld + column(c), n - column(c), row::pack<KIND>(v[c]));
    }
  }
}

constexpr int kSms = 152;

template <int KIND, bool WIDE, int C, int THREADS>
cudaError_t launch_rows(const RowParams& p, const ff::LaunchShape& shape, cudaStream_t stream) {
  static_assert(5 * C * THREADS * 16 <= 160 * 1024, "the parameters' words");
  cudaError_t e = prepare_smem<row_forward_kernel<KIND, WIDE, C, THREADS>>(5 * C * THREADS * 16);
  return e != cudaSuccess ? e : ff::launch_early(stream, shape, row_forward_kernel<KIND, WIDE, C, THREADS>, p);
}

template <int KIND, int C, int THREADS>
cudaError_t run_rows(const ForwardTask& t, int threads, cudaStream_t stream) {
  RowParams p;
  bool wide = true;
  p.x = row::view_of(t.X.p, t.X.ld, t.M, t.N), p.h = row::view_of(t.H.p, t.H.ld, t.M, t.N);
  p.r = row::view_of(t.R.p, t.R.ld, t.M, t.N), p.y = row::view_of(t.Y.p, t.Y.ld, t.M, t.N);
  const uint16_t* const vectors[5] = {t.post_weight, t.post_bias, t.gate.p, t.weight, t.bias};
  int slots = 0;
  for (int i = 0; i < 5; ++i) {
    const int64_t rows = i == kGate ? t.gates : 1;
    p.vector[i] = row::view_of(vectors[i], t.gate.ld, rows, t.N);
    wide = wide && row::whole_words(p.vector[i], t.N);
    p.slot[i] = vectors[i] != nullptr && rows == 1 ? slots++ : -1;
  }
  for (const row::View& v : {p.x, p.h, p.r, p.y}) wide = wide && row::whole_words(v, t.N);
  p.M = t.M, p.rows_per_gate = t.M / t.gates, p.N = static_cast<int>(t.N), p.threads = threads;
  p.norm = t.norm, p.post = t.post, p.scale = t.scale, p.eps = t.eps, p.drop = t.drop;
  const int rows = THREADS / threads;
  const int64_t blocks = (t.M + rows - 1) / rows, most = kSms * blocks_of<C, THREADS>();
  const ff::LaunchShape shape{dim3(static_cast<unsigned>(blocks < most ? blocks : most)), rows * threads, 1,
                              slots * C * rows * threads * 16};
  return wide ? launch_rows<KIND, true, C, THREADS>(p, shape, stream) : launch_rows<KIND, false, C, THREADS>(p, shape, stream);
}

// A row of up to 1024 values by one warp (no barriers), up to 8192 in two words a thread, up to 16384 with as many
// threads as a block has; longer ones in passes over memory.
template <int KIND>
cudaError_t run(const ForwardTask& t, cudaStream_t stream) {
  const int64_t words = (t.N + row::kWord - 1) / row::kWord;
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
