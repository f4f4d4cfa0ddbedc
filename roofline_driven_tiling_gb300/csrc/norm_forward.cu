// norm_forward.cu -- r = scale x + gate drop(post(h)), y = norm(r).
//
// x and h are read once and r and y written once where a row fits the registers of a block (N <= 8192): mean first, then
// the squares of what is left of it. A warp takes a row of up to 1024 values alone, without barriers; longer ones take two
// words a thread. The next row's words come to shared memory behind this row's sums, also where rows start off 16-byte
// boundaries. Bound by memory: 8192 x 4096 with a second norm 44.4 us (6.0 TB/s), 4096 x 8192 46; one row of 4096 2.6 us (the
// launch). 8192 x 1003 off boundaries 42 us (8192 x 1000 13), bound by the instructions that put words together. Rows beyond
// 8192 take passes over memory of two bytes a load: 4096 x 12288 225 us (1.8 TB/s), without h 71; one row of 16384 11.
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

// Rows of up to 8192 values: a group of threads keeps a row in registers, C words of eight values a thread. The next
// row's words come to shared memory meanwhile, and the parameters' words stay there; a thread reads what it fetched itself.
enum Place : int { kX = 0, kH = 1, kPostWeight = 2, kPostBias = 3, kGate = 4, kWeight = 5, kBias = 6, kPlaces = 7 };
struct RowParams {
  row::View in[kPlaces], r, y;
  int at[kPlaces];  // of its words in shared memory, in bytes; -1: absent, or a gate that changes
  int64_t M, rows_per_gate, step;  // rows that all groups take at once
  int64_t inner_end;  // of the rows of x and h whose aligned words lie within both
  int64_t x_step, h_step, r_step, y_step;
  int N, threads;  // threads of a row
  int norm, post;
  float scale, eps;
  Dropout drop;
};

// Blocks that an SM holds: 64 registers a thread, four words a thread twice as many.
template <int C, int THREADS>
constexpr int blocks_of() {
  return (C == 4 ? 512 : 1024) / THREADS;
}

template <int KIND, bool WIDE, int C, int THREADS>
__global__ void __launch_bounds__(THREADS, blocks_of<C, THREADS>()) row_forward_kernel(const __grid_constant__ RowParams p) {
  extern __shared__ uint4 words[];
  __shared__ float rooms[row::Group::kRoomFloats];
  constexpr uint32_t kPitch = THREADS / 32 * row::kWarpBytes<WIDE>;  // in shared memory, from one of a thread's words to the next
  ff::wait_for_earlier_kernels();
  row::Group group(p.threads, rooms);
  const int n = p.N, rows_at_once = static_cast<int>(blockDim.x) / p.threads;
  const uint64_t groups = static_cast<uint64_t>((static_cast<int64_t>(n) + 3) / 4);
  const float inv_n = 1.0f / static_cast<float>(n);
  const uint64_t key = p.drop.dropped != 0 ? drop_key(p.drop) : 0;
  const bool has_h = p.in[kH].p != nullptr;
  const int first = group.rank * row::kWord, stride = p.threads * row::kWord;
  auto left = [&](int c) { return n - first - c * stride; };
  const uint32_t mine = smem_u32(words) + row::place_of_thread<WIDE>();
  auto fetch = [&](int place, const uint16_t* from, bool inside) {
#pragma unroll
    for (int c = 0; c < C; ++c)
      row::fetch_word<WIDE>(mine + p.at[place] + c * kPitch, p.in[place], from + c * stride, left(c), inside);
  };
  auto settle = [&](int place, const uint16_t* from) {
#pragma unroll
    for (int c = 0; c < C; ++c) row::settle<WIDE>(mine + p.at[place] + c * kPitch, from + c * stride, left(c));
  };
  auto get = [&](int place, int c, uint64_t(&f)[4]) {
    row::unpack<KIND>(row::arrived<WIDE>(mine + p.at[place] + c * kPitch, left(c)), f);
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
        row::clear_from<WIDE>(v[c], left(c));
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
    if (p.at[weight] >= 0) {
      get(weight, c, w);
#pragma unroll
      for (int i = 0; i < 4; ++i) v[c][i] = row::mul2(v[c][i], w[i]);
    }
    if (p.at[bias] >= 0) {
      get(bias, c, w);
#pragma unroll
      for (int i = 0; i < 4; ++i) v[c][i] = row::add2(v[c][i], w[i]);
    }
  };

  int64_t m = static_cast<int64_t>(blockIdx.x) * rows_at_once + group.index;
  const uint16_t* x = p.in[kX].p + m * p.in[kX].ld + first;
  const uint16_t* h = p.in[kH].p + m * p.in[kH].ld + first;
  uint16_t* r = p.r.p + m * p.r.ld + first;
  uint16_t* y = p.y.p + m * p.y.ld + first;
#pragma unroll 1
  for (int i = 0; i < kPlaces; ++i)
    if (p.at[i] >= 0)
#pragma unroll
      for (int c = 0; c < C; ++c) row::clear_place<WIDE>(mine + p.at[i] + c * kPitch, left(c));
#pragma unroll 1
  for (int i = kPostWeight; i < kPlaces; ++i)
    if (p.at[i] >= 0) fetch(i, p.in[i].p + first, false);
  if (m < p.M) {
    fetch(kX, x, false);
    if (has_h) fetch(kH, h, false);
  }
  if (!WIDE) {
    row::wait_copies();
#pragma unroll 1
    for (int i = kPostWeight; i < kPlaces; ++i)
      if (p.at[i] >= 0) settle(i, p.in[i].p + first);
  }
  for (; m < p.M; m += p.step, x += p.x_step, h += p.h_step, r += p.r_step, y += p.y_step) {
    const bool more = m + p.step < p.M, inside = m + p.step < p.inner_end;  // the next row
    row::wait_copies();
    settle(kX, x);
    if (has_h) {
      settle(kH, h);
#pragma unroll
      for (int c = 0; c < C; ++c) get(kH, c, v[c]);
      if (more) fetch(kH, h + p.h_step, inside);
      const float rstd = p.post != T2S_NORM_NONE ? scale_of(p.post) : 1.0f;
#pragma unroll
      for (int c = 0; c < C; ++c) {
        uint64_t u[4];
        if (p.post != T2S_NORM_NONE) affine(rstd, kPostWeight, kPostBias, c);
        if (p.drop.dropped != 0) {
          row::Keep keep;
          keep.draw(key, static_cast<uint64_t>(m) * groups + static_cast<uint64_t>((first + c * stride) / 4), p.drop.dropped);
          keep.apply(v[c], p.drop.factor);
        }
        if (p.in[kGate].p != nullptr) {
          if (p.at[kGate] >= 0) {
            get(kGate, c, u);
          } else {
            const uint16_t* gate = p.in[kGate].p + m / p.rows_per_gate * p.in[kGate].ld + first + c * stride;
            row::unpack<KIND>(row::load_word<WIDE>(p.in[kGate], gate, left(c)), u);
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) v[c][i] = row::mul2(v[c][i], u[i]);
        }
        get(kX, c, u);
#pragma unroll
        for (int i = 0; i < 4; ++i) v[c][i] = row::fma2(u[i], row::both(p.scale), v[c][i]);
        // The norm that follows is of the rounded values.
        const uint4 rounded = row::pack<KIND>(v[c]);
        row::store_word<WIDE>(p.r, r + c * stride, left(c), rounded);
        row::unpack<KIND>(rounded, v[c]);
        row::clear_from<WIDE>(v[c], left(c));
      }
    } else {
#pragma unroll
      for (int c = 0; c < C; ++c) get(kX, c, v[c]);
    }
    if (more) fetch(kX, x + p.x_step, inside);
    if (p.norm == T2S_NORM_NONE) continue;
    const float rstd = scale_of(p.norm);
#pragma unroll
    for (int c = 0; c < C; ++c) {
      affine(rstd, kWeight, kBias, c);
      row::store_word<WIDE>(p.y, y + c * stride, left(c), row::pack<KIND>(v[c]));
    }
  }
  row::wait_copies();  // a group without a row has waited for none: its parameters' copies land before the CTA's memory goes
}

constexpr int kSms = 152, kMostSmem = 226 * 1024;

template <int KIND, bool WIDE, int C, int THREADS>
cudaError_t launch_rows(RowParams& p, int block, cudaStream_t stream) {
  constexpr int kSlot = C * (THREADS / 32) * static_cast<int>(row::kWarpBytes<WIDE>);
  static_assert(kPlaces * kSlot <= kMostSmem, "shared memory of one CTA");
  int used = 0;
  for (int i = 0; i < kPlaces; ++i)
    if (p.at[i] >= 0) {
      p.at[i] = used;
      used += kSlot;
    }
  cudaError_t e = prepare_smem<row_forward_kernel<KIND, WIDE, C, THREADS>>(kPlaces * kSlot);
  if (e != cudaSuccess) return e;
  // As many blocks as the SMs hold, by registers and by shared memory.
  const int by_smem = kMostSmem / (used + 2048), held = by_smem < blocks_of<C, THREADS>() ? by_smem : blocks_of<C, THREADS>();
  const int64_t most = static_cast<int64_t>(kSms) * held;
  const int64_t at_once = block / p.threads, blocks = (p.M + at_once - 1) / at_once;
  const int grid = static_cast<int>(blocks < most ? blocks : most);
  p.step = grid * at_once;
  p.x_step = p.step * p.in[kX].ld, p.h_step = p.step * p.in[kH].ld, p.r_step = p.step * p.r.ld, p.y_step = p.step * p.y.ld;
  return ff::launch_early(stream, {dim3(static_cast<unsigned>(grid)), block, 1, used},
                          row_forward_kernel<KIND, WIDE, C, THREADS>, p);
}

template <int KIND, int C, int THREADS>
cudaError_t run_rows(const ForwardTask& t, int threads, cudaStream_t stream) {
  RowParams p;
  bool wide = true;
  const uint16_t* const inputs[kPlaces] = {t.X.p, t.H.p, t.post_weight, t.post_bias, t.gate.p, t.weight, t.bias};
  const int64_t ld[kPlaces] = {t.X.ld, t.H.ld, 0, 0, t.gate.ld, 0, 0}, rows[kPlaces] = {t.M, t.M, 1, 1, t.gates, 1, 1};
  for (int i = 0; i < kPlaces; ++i) {
    p.in[i] = row::view_of(inputs[i], ld[i], rows[i], t.N);
    p.at[i] = inputs[i] != nullptr && (i != kGate || t.gates == 1) ? 0 : -1;
    wide = wide && row::whole_words(p.in[i], t.N);
  }
  p.r = row::view_of(t.R.p, t.R.ld, t.M, t.N), p.y = row::view_of(t.Y.p, t.Y.ld, t.M, t.N);
  wide = wide && row::whole_words(p.r, t.N) && row::whole_words(p.y, t.N);
  const int64_t x_end = row::inner_end(p.in[kX], t.M), h_end = row::inner_end(p.in[kH], t.M);
  p.inner_end = x_end < h_end ? x_end : h_end;
  p.M = t.M, p.rows_per_gate = t.M / t.gates, p.N = static_cast<int>(t.N), p.threads = threads;
  p.norm = t.norm, p.post = t.post, p.scale = t.scale, p.eps = t.eps, p.drop = t.drop;
  const int block = THREADS / threads * threads;
  return wide ? launch_rows<KIND, true, C, THREADS>(p, block, stream) : launch_rows<KIND, false, C, THREADS>(p, block, stream);
}

// A row of up to 1024 values by one warp (no barriers), up to 8192 in two words a thread; longer ones in passes over
// memory.
template <int KIND>
cudaError_t run(const ForwardTask& t, cudaStream_t stream) {
  const int64_t words = (t.N + row::kWord - 1) / row::kWord;
  if (words <= 32) return run_rows<KIND, 1, 256>(t, 32, stream);
  if (words <= 64) return run_rows<KIND, 2, 256>(t, 32, stream);
  if (words <= 128) return run_rows<KIND, 4, 256>(t, 32, stream);
  const int threads = static_cast<int>((words + 63) / 64 * 32);
  if (threads <= 256) return run_rows<KIND, 2, 256>(t, threads, stream);
  if (threads <= 512) return run_rows<KIND, 2, 512>(t, threads, stream);
  const unsigned blocks = static_cast<unsigned>(t.M < 2 * kSms ? t.M : 2 * kSms);
  return ff::launch_early(stream, {dim3(blocks), kWideThreads, 1, 0}, wide_forward_kernel<KIND>, t);
}

}  // namespace

cudaError_t run_forward(const ForwardTask& t, cudaStream_t stream) {
  return t.kind == ff::kBf16 ? run<ff::kBf16>(t, stream) : run<ff::kF16>(t, stream);
}

}  // namespace norm
}  // namespace t2s
