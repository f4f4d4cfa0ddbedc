// norm_backward.cu -- the gradients of r = scale x + gate drop(post(h)), y = norm(r).
//
// With xh = (r - mean) rho, g = dy weight, and the same for h (hh, sigma) and its gradient:
//   d = dr + rho (g - [mean g] - xh mean(g xh)),  [mean g] for layer norms only;  dx = scale d
//   dn = drop'(d gate),  q = dn post_weight,  dh = sigma (q - [mean q] - hh mean(q hh))
//   dweight = sum dy xh, dbias = sum dy, dgate = sum d drop(n), dpost_weight = sum dn hh, dpost_bias = sum dn
// A CTA takes consecutive rows and adds its rows' share of the five sums in FP32; a second launch adds the
// CTAs' shares in their order.
#include <cuda_runtime.h>

#include <cstdint>
#include <cstring>

#include "matrix_args.h"
#include "norm_device.cuh"

namespace t2s {
namespace norm {
namespace {

constexpr int kWideThreads = 1024;
constexpr int kVectors = 5;
enum Vector : int { kWeight = 0, kBias = 1, kGate = 2, kPostWeight = 3, kPostBias = 4 };

// How the rows lie on the CTAs. Few gates: `pieces` CTAs to each gate's rows. Otherwise a CTA takes whole
// gates (and one gate's sum is complete when its rows are).
struct Split {
  int ctas, pieces;  // pieces 0: whole gates
};
constexpr int kMostCtas = 304;
Split split_of(int64_t M, int64_t gates) {
  const int64_t rows = M / gates;
  if (2 * gates > kMostCtas) return {static_cast<int>(gates < kMostCtas ? gates : kMostCtas), 0};
  int64_t pieces = kMostCtas / gates;
  if (pieces > rows) pieces = rows;
  return {static_cast<int>(gates * pieces), static_cast<int>(pieces)};
}

struct BackwardParams {
  BackwardTask t;
  Split split;
  int slot[kVectors];  // of a CTA's partial sums; -1: not wanted
  int slots;
};

// The rows of CTA c, and those of one gate after another among them.
struct Rows {
  int64_t first, last, per_gate;
};
__device__ __forceinline__ Rows rows_of(const BackwardParams& p, int64_t c) {
  const int64_t per_gate = p.t.M / p.t.gates;
  if (p.split.pieces > 0) {
    const int64_t g = c / p.split.pieces, j = c % p.split.pieces;
    return {g * per_gate + per_gate * j / p.split.pieces, g * per_gate + per_gate * (j + 1) / p.split.pieces, per_gate};
  }
  return {p.t.gates * c / p.split.ctas * per_gate, p.t.gates * (c + 1) / p.split.ctas * per_gate, per_gate};
}

// Rows of any length: passes over memory, the partial sums in memory too (each value belongs to one thread).
template <int KIND>
__global__ void __launch_bounds__(kWideThreads) wide_backward_kernel(const __grid_constant__ BackwardParams p) {
  __shared__ float room[96];
  ff::wait_for_earlier_kernels();
  const BackwardTask& t = p.t;
  const int64_t groups = (t.N + 3) / 4;
  const float inv_n = 1.0f / static_cast<float>(t.N);
  const uint64_t key = t.drop.dropped != 0 ? drop_key(t.drop) : 0;
  const Rows rows = rows_of(p, blockIdx.x);
  float* const partials = t.partials + static_cast<int64_t>(blockIdx.x) * p.slots * t.N;
  const bool has_h = t.H.p != nullptr;
  for (int64_t m = rows.first; m < rows.last; ++m) {
    const bool first = m == rows.first, gate_first = p.split.pieces > 0 ? first : m % rows.per_gate == 0;
    const bool gate_last = p.split.pieces == 0 && (m + 1) % rows.per_gate == 0;
    const uint16_t* r = t.R.p + m * t.R.ld;
    const uint16_t* dy = t.dY.p + m * t.dY.ld;
    const uint16_t* dr = t.dR.p == nullptr ? nullptr : t.dR.p + m * t.dR.ld;
    const uint16_t* h = t.H.p + m * t.H.ld;
    const uint16_t* gate = t.gate.p == nullptr ? nullptr : t.gate.p + m / rows.per_gate * t.gate.ld;
    float mean = 0.0f, rho = 1.0f, mean_g = 0.0f, mean_gx = 0.0f;
    if (t.norm == T2S_NORM_LAYER) {
      float s[1] = {0.0f};
      for (int64_t n = threadIdx.x; n < t.N; n += kWideThreads) s[0] += ff::to_f32<KIND>(r[n]);
      block_sums(s, room);
      mean = s[0] * inv_n;
    }
    if (t.norm != T2S_NORM_NONE) {
      float s[3] = {};
      for (int64_t n = threadIdx.x; n < t.N; n += kWideThreads) {
        const float c = ff::to_f32<KIND>(r[n]) - mean, g = ff::to_f32<KIND>(dy[n]) * at<KIND>(t.weight, n, 1.0f);
        s[0] = fmaf(c, c, s[0]);
        s[1] += g;
        s[2] = fmaf(g, c, s[2]);
      }
      block_sums(s, room);
      rho = rsqrtf(s[0] * inv_n + t.eps);
      mean_g = t.norm == T2S_NORM_LAYER ? s[1] * inv_n : 0.0f;
      mean_gx = s[2] * inv_n * rho;
    }
    float h_mean = 0.0f, sigma = 1.0f;
    if (has_h && t.post == T2S_NORM_LAYER) {
      float s[1] = {0.0f};
      for (int64_t n = threadIdx.x; n < t.N; n += kWideThreads) s[0] += ff::to_f32<KIND>(h[n]);
      block_sums(s, room);
      h_mean = s[0] * inv_n;
    }
    if (has_h && t.post != T2S_NORM_NONE) {
      float s[1] = {0.0f};
      for (int64_t n = threadIdx.x; n < t.N; n += kWideThreads) {
        const float c = ff::to_f32<KIND>(h[n]) - h_mean;
        s[0] = fmaf(c, c, s[0]);
      }
      block_sums(s, room);
      sigma = rsqrtf(s[0] * inv_n + t.eps);
    }
    // d at a column, from memory each time.
    auto gradient = [&](int64_t n) {
      float d = at<KIND>(dr, n, 0.0f);
      if (t.norm != T2S_NORM_NONE) {
        const float xh = (ff::to_f32<KIND>(r[n]) - mean) * rho, g = ff::to_f32<KIND>(dy[n]) * at<KIND>(t.weight, n, 1.0f);
        d += rho * (g - mean_g - xh * mean_gx);
      }
      return d;
    };
    auto add = [&](int vector, int64_t n, float v, bool start) {
      if (p.slot[vector] < 0) return;
      float* to = partials + p.slot[vector] * t.N + n;
      *to = start ? v : *to + v;
    };
    float s[2] = {};
    for (int64_t n = threadIdx.x; n < t.N; n += kWideThreads) {
      const float d = gradient(n);
      if (t.norm != T2S_NORM_NONE) {
        const float y = ff::to_f32<KIND>(dy[n]);
        add(kWeight, n, y * ((ff::to_f32<KIND>(r[n]) - mean) * rho), first);
        add(kBias, n, y, first);
      }
      if (t.dX.p != nullptr) t.dX.p[m * t.dX.ld + n] = ff::from_f32<KIND>(t.scale * d);
      if (!has_h) continue;
      const float hh = (ff::to_f32<KIND>(h[n]) - h_mean) * sigma, pw = at<KIND>(t.post_weight, n, 1.0f);
      float v = t.post == T2S_NORM_NONE ? hh : fmaf(hh, pw, at<KIND>(t.post_bias, n, 0.0f));
      float dn = d * at<KIND>(gate, n, 1.0f);
      if (t.drop.dropped != 0) {
        const uint64_t bits = drop_bits(key, static_cast<uint64_t>(m * groups + n / 4));
        v = drop(v, bits, n & 3, t.drop.dropped, t.drop.factor);
        dn = drop(dn, bits, n & 3, t.drop.dropped, t.drop.factor);
      }
      add(kGate, n, d * v, gate_first);
      if (gate_last && p.slot[kGate] >= 0)
        t.dgate.p[m / rows.per_gate * t.dgate.ld + n] = ff::from_f32<KIND>(partials[p.slot[kGate] * t.N + n]);
      if (t.post == T2S_NORM_NONE) {
        if (t.dH.p != nullptr) t.dH.p[m * t.dH.ld + n] = ff::from_f32<KIND>(dn);
        continue;
      }
      add(kPostWeight, n, dn * hh, first);
      add(kPostBias, n, dn, first);
      s[0] += dn * pw;
      s[1] = fmaf(dn * pw, hh, s[1]);
    }
    if (!has_h || t.post == T2S_NORM_NONE || t.dH.p == nullptr) continue;
    block_sums(s, room);
    const float mean_q = t.post == T2S_NORM_LAYER ? s[0] * inv_n : 0.0f, mean_qh = s[1] * inv_n;
    for (int64_t n = threadIdx.x; n < t.N; n += kWideThreads) {
      float dn = gradient(n) * at<KIND>(gate, n, 1.0f);
      if (t.drop.dropped != 0)
        dn = drop(dn, drop_bits(key, static_cast<uint64_t>(m * groups + n / 4)), n & 3, t.drop.dropped, t.drop.factor);
      const float hh = (ff::to_f32<KIND>(h[n]) - h_mean) * sigma;
      t.dH.p[m * t.dH.ld + n] =
          ff::from_f32<KIND>(sigma * (dn * at<KIND>(t.post_weight, n, 1.0f) - mean_q - hh * mean_qh));
    }
  }
}

// Adds the CTAs' shares: a block takes 32 columns of one vector (or of one row of dgate), its warps every
// kSumWarps-th share each.
constexpr int kSumWarps = 16;
struct SumParams {
  const float* partials;
  int64_t N, ldgate;
  uint16_t* out[kVectors];
  int slot[kVectors];
  int slots, ctas, pieces, vectors, gate_rows;
};

template <int KIND>
__global__ void __launch_bounds__(32 * kSumWarps) share_sum_kernel(const __grid_constant__ SumParams p) {
  __shared__ float room[kSumWarps][33];
  ff::wait_for_earlier_kernels();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // Vectors other than the gate first, then the gate's rows.
  int v = static_cast<int>(blockIdx.y), first = 0, last = p.ctas;
  int64_t row = 0;
  if (v >= p.vectors) {
    row = v - p.vectors;
    v = kGate;
    first = static_cast<int>(row) * p.pieces, last = first + p.pieces;
  }
  const int64_t n = static_cast<int64_t>(blockIdx.x) * 32 + lane;
  // The slot's vector: the v-th wanted one that is not the gate.
  int which = v;
  if (static_cast<int>(blockIdx.y) < p.vectors) {
    which = 0;
    for (int left = v; which < kVectors; ++which) {
      if (which == kGate || p.slot[which] < 0) continue;
      if (left-- == 0) break;
    }
  }
  float sum = 0.0f;
  if (n < p.N)
#pragma unroll 4
    for (int c = first + warp; c < last; c += kSumWarps)
      sum += p.partials[(static_cast<int64_t>(c) * p.slots + p.slot[which]) * p.N + n];
  room[warp][lane] = sum;
  __syncthreads();
  if (warp != 0 || n >= p.N) return;
  for (int i = 1; i < kSumWarps; ++i) sum += room[i][lane];
  p.out[which][row * p.ldgate + n] = ff::from_f32<KIND>(sum);
}

template <int KIND>
cudaError_t run(const BackwardTask& t, cudaStream_t stream) {
  BackwardParams p;
  p.t = t;
  p.split = split_of(t.M, t.gates);
  uint16_t* const outs[kVectors] = {t.dweight, t.dbias, t.dgate.p, t.dpost_weight, t.dpost_bias};
  p.slots = 0;
  SumParams s;
  memset(&s, 0, sizeof(s));
  for (int i = 0; i < kVectors; ++i) {
    p.slot[i] = s.slot[i] = outs[i] != nullptr ? p.slots++ : -1;
    s.out[i] = outs[i];
    if (i != kGate && outs[i] != nullptr) ++s.vectors;
  }
  if (p.slots == 0 && t.dX.p == nullptr && t.dH.p == nullptr) return cudaSuccess;
  cudaError_t e = ff::launch_early(stream, {dim3(static_cast<unsigned>(p.split.ctas)), kWideThreads, 1, 0},
                                   wide_backward_kernel<KIND>, p);
  if (e != cudaSuccess) return e;
  s.gate_rows = t.dgate.p != nullptr && p.split.pieces > 0 ? static_cast<int>(t.gates) : 0;
  if (s.vectors + s.gate_rows == 0) return cudaSuccess;
  s.partials = t.partials;
  s.N = t.N;
  s.ldgate = t.dgate.ld;
  s.slots = p.slots;
  s.ctas = p.split.ctas;
  s.pieces = p.split.pieces;
  const dim3 grid(static_cast<unsigned>((t.N + 31) / 32), static_cast<unsigned>(s.vectors + s.gate_rows));
  return ff::launch_early(stream, {grid, 32 * kSumWarps, 1, 0}, share_sum_kernel<KIND>, s);
}

}  // namespace

size_t backward_workspace_bytes(int64_t M, int64_t N, int64_t gates, int vectors) {
  if (M == 0 || N == 0 || vectors == 0) return 0;
  return static_cast<size_t>(split_of(M, gates).ctas) * static_cast<size_t>(vectors) * static_cast<size_t>(N) * 4;
}

cudaError_t run_backward(const BackwardTask& t, cudaStream_t stream) {
  return t.kind == ff::kBf16 ? run<ff::kBf16>(t, stream) : run<ff::kF16>(t, stream);
}

}  // namespace norm
}  // namespace t2s
