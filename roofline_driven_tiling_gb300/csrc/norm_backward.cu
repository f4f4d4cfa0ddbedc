// norm_backward.cu -- the gradients of r = scale x + gate drop(post(h)), y = norm(r).
//
// With xh = (r - mean) rho, g = dy weight, and the same for h (hh, sigma) and its gradient:
//   d = dr + rho (g - [mean g] - xh mean(g xh)),  [mean g] for layer norms only;  dx = scale d
//   dn = drop'(d gate),  q = dn post_weight,  dh = sigma (q - [mean q] - hh mean(q hh))
//   dweight = sum dy xh, dbias = sum dy, dgate = sum d drop(n), dpost_weight = sum dn hh, dpost_bias = sum dn
// A CTA takes consecutive rows and adds its rows' share of the five sums in FP32; a second launch adds the
// CTAs' shares in their order.
#include <cuda_runtime.h>

#include <atomic>
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

// Rows of up to 8192 values: a group of threads keeps a row in registers, a word of eight values a thread; a block
// holds several groups. The sums over rows are added in shared memory, each group's in its own place, every value by
// one thread; at the end of a block's rows (of a gate's for dgate) the groups' sums are added in their order.
struct RowParams {
  BackwardParams b;
  int threads;  // of a row
  int dy_wide, dr_wide, r_wide, h_wide, dx_wide, dh_wide, gate_wide, vectors_wide;
};

template <int KIND, int THREADS>
__global__ void __launch_bounds__(THREADS, 1024 / THREADS) row_backward_kernel(const __grid_constant__ RowParams p) {
  extern __shared__ float sums[];  // slots x N for each group
  __shared__ float rooms[Group::kRoomFloats];
  const BackwardTask& t = p.b.t;
  Group group(p.threads, rooms);
  const int n = static_cast<int>(t.N), slots = p.b.slots, rows_at_once = static_cast<int>(blockDim.x) / p.threads;
  const int pitch = (n + kWord - 1) / kWord * kWord;
  float* const mine = sums + static_cast<int64_t>(group.index) * slots * pitch;
  for (int i = threadIdx.x; i < rows_at_once * slots * pitch; i += blockDim.x) sums[i] = 0.0f;
  __syncthreads();
  ff::wait_for_earlier_kernels();
  const int64_t groups = (t.N + 3) / 4;
  const float inv_n = 1.0f / static_cast<float>(n);
  const uint64_t key = t.drop.dropped != 0 ? drop_key(t.drop) : 0;
  const bool has_h = t.H.p != nullptr, has_norm = t.norm != T2S_NORM_NONE, has_post = has_h && t.post != T2S_NORM_NONE;
  const bool layer = t.norm == T2S_NORM_LAYER, post_layer = has_post && t.post == T2S_NORM_LAYER;
  const Rows rows = rows_of(p.b, blockIdx.x);
  const int at = group.rank * kWord, left = n - at;
  auto add = [&](int vector, const float (&v)[kWord]) {
    if (p.b.slot[vector] < 0) return;
    float4* to = reinterpret_cast<float4*>(mine + p.b.slot[vector] * pitch + at);
    float4 a = to[0], b = to[1];
    a.x += v[0], a.y += v[1], a.z += v[2], a.w += v[3];
    b.x += v[4], b.y += v[5], b.z += v[6], b.w += v[7];
    to[0] = a, to[1] = b;
  };
  // One gate's rows after another (one stretch of rows where a gate has several blocks).
  const int64_t stretch = p.b.split.pieces > 0 ? rows.last - rows.first : rows.per_gate;
  for (int64_t m0 = rows.first; m0 < rows.last; m0 += stretch) {
    const int64_t gate_row = m0 / rows.per_gate;
    const uint16_t* gate = t.gate.p == nullptr ? nullptr : t.gate.p + gate_row * t.gate.ld;
    for (int64_t m = m0 + group.index; m < m0 + stretch; m += rows_at_once) {
      uint4 r4 = make_uint4(0, 0, 0, 0), dy4 = r4, dr4 = r4, h4 = r4;
      if (left > 0) {
        if (has_norm) {
          r4 = load_word(t.R.p + m * t.R.ld + at, left, p.r_wide);
          dy4 = load_word(t.dY.p + m * t.dY.ld + at, left, p.dy_wide);
        }
        if (t.dR.p != nullptr) dr4 = load_word(t.dR.p + m * t.dR.ld + at, left, p.dr_wide);
        if (has_h) h4 = load_word(t.H.p + m * t.H.ld + at, left, p.h_wide);
      }
      float xh[kWord], g[kWord], hh[kWord];
      unpack<KIND>(r4, xh);
      unpack<KIND>(h4, hh);
      float means[2] = {0.0f, 0.0f};
      if (layer || post_layer) {
#pragma unroll
        for (int i = 0; i < kWord; ++i) means[0] += xh[i], means[1] += hh[i];
        group.sums(means);
        means[0] = layer ? means[0] * inv_n : 0.0f;
        means[1] = post_layer ? means[1] * inv_n : 0.0f;
#pragma unroll
        for (int i = 0; i < kWord; ++i)
          if (i < left) xh[i] -= means[0], hh[i] -= means[1];
      }
      unpack<KIND>(dy4, g);
      float w[kWord];
      if (left > 0 && t.weight != nullptr) {
        parameter<KIND>(t.weight, at, left, p.vectors_wide, 1.0f, w);
#pragma unroll
        for (int i = 0; i < kWord; ++i) g[i] *= w[i];
      }
      float s[4] = {};
#pragma unroll
      for (int i = 0; i < kWord; ++i) {
        s[0] = fmaf(xh[i], xh[i], s[0]);
        s[1] += g[i];
        s[2] = fmaf(g[i], xh[i], s[2]);
        s[3] = fmaf(hh[i], hh[i], s[3]);
      }
      if (has_norm || has_post) group.sums(s);
      const float rho = rsqrtf(s[0] * inv_n + t.eps), sigma = has_post ? rsqrtf(s[3] * inv_n + t.eps) : 1.0f;
      const float mean_g = layer ? s[1] * inv_n : 0.0f, mean_gx = s[2] * inv_n * rho;
      float d[kWord];
      unpack<KIND>(dr4, d);
      if (has_norm) {
#pragma unroll
        for (int i = 0; i < kWord; ++i) {
          xh[i] *= rho;
          d[i] += rho * (g[i] - mean_g - xh[i] * mean_gx);
          if (i >= left) d[i] = 0.0f;  // the means are not for the values beyond the row's end
        }
      }
      float q[2] = {0.0f, 0.0f};
      if (left > 0) {
        if (has_norm) {
          unpack<KIND>(dy4, g);
          add(kBias, g);
#pragma unroll
          for (int i = 0; i < kWord; ++i) g[i] *= xh[i];
          add(kWeight, g);
        }
        if (t.dX.p != nullptr) {
#pragma unroll
          for (int i = 0; i < kWord; ++i) g[i] = t.scale * d[i];
          store_word(t.dX.p + m * t.dX.ld + at, left, p.dx_wide, pack<KIND>(g));
        }
        if (has_h) {
          float pw[kWord];
          parameter<KIND>(t.post_weight, at, left, p.vectors_wide, 1.0f, pw);
#pragma unroll
          for (int i = 0; i < kWord; ++i) hh[i] *= sigma;
          const uint64_t word = static_cast<uint64_t>(m * groups + at / 4);
          if (p.b.slot[kGate] >= 0) {
            if (has_post) {
              parameter<KIND>(t.post_bias, at, left, p.vectors_wide, 0.0f, w);
#pragma unroll
              for (int i = 0; i < kWord; ++i) g[i] = fmaf(hh[i], pw[i], w[i]);
            } else {
#pragma unroll
              for (int i = 0; i < kWord; ++i) g[i] = hh[i];
            }
            if (t.drop.dropped != 0) drop_word(t.drop, key, word, g);
#pragma unroll
            for (int i = 0; i < kWord; ++i) g[i] *= d[i];
            add(kGate, g);
          }
          if (gate != nullptr) {
            parameter<KIND>(gate, at, left, p.gate_wide, 1.0f, w);
#pragma unroll
            for (int i = 0; i < kWord; ++i) d[i] *= w[i];
          }
          if (t.drop.dropped != 0) drop_word(t.drop, key, word, d);
          if (has_post) {
            add(kPostBias, d);
#pragma unroll
            for (int i = 0; i < kWord; ++i) g[i] = d[i] * hh[i];
            add(kPostWeight, g);
#pragma unroll
            for (int i = 0; i < kWord; ++i) {
              d[i] *= pw[i];
              q[0] += d[i];
              q[1] = fmaf(d[i], hh[i], q[1]);
            }
          }
        }
      }
      if (!has_h || t.dH.p == nullptr) continue;
      if (has_post) {
        group.sums(q);
        const float mean_q = post_layer ? q[0] * inv_n : 0.0f, mean_qh = q[1] * inv_n;
#pragma unroll
        for (int i = 0; i < kWord; ++i) d[i] = sigma * (d[i] - mean_q - hh[i] * mean_qh);
      }
      if (left > 0) store_word(t.dH.p + m * t.dH.ld + at, left, p.dh_wide, pack<KIND>(d));
    }
    if (p.b.split.pieces == 0 && p.b.slot[kGate] >= 0) {
      __syncthreads();
      for (int i = threadIdx.x; i < n; i += blockDim.x) {
        float sum = 0.0f;
        for (int j = 0; j < rows_at_once; ++j) {
          float* from = sums + (static_cast<int64_t>(j) * slots + p.b.slot[kGate]) * pitch + i;
          sum += *from;
          *from = 0.0f;
        }
        t.dgate.p[gate_row * t.dgate.ld + i] = ff::from_f32<KIND>(sum);
      }
      __syncthreads();
    }
  }
  __syncthreads();
  float* const out = t.partials + static_cast<int64_t>(blockIdx.x) * slots * n;
  for (int slot = 0; slot < slots; ++slot)
    for (int i = threadIdx.x; i < n; i += blockDim.x) {
      float sum = 0.0f;
      for (int j = 0; j < rows_at_once; ++j) sum += sums[(static_cast<int64_t>(j) * slots + slot) * pitch + i];
      out[static_cast<int64_t>(slot) * n + i] = sum;
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

template <int KIND, int THREADS>
cudaError_t launch_rows(const BackwardParams& b, cudaStream_t stream) {
  constexpr int kMaxDevices = 64, kMaxSmem = 5 * 8192 * 4;
  static std::atomic<bool> prepared[kMaxDevices];
  auto kern = row_backward_kernel<KIND, THREADS>;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
  if (!prepared[dev].load(std::memory_order_acquire)) {
    if ((e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxSmem)) != cudaSuccess) return e;
    prepared[dev].store(true, std::memory_order_release);
  }
  const BackwardTask& t = b.t;
  const int words = static_cast<int>((t.N + kWord - 1) / kWord);
  RowParams p{b, (words + 31) / 32 * 32};
  p.dy_wide = wide_rows(t.dY.p, t.dY.ld, t.M), p.dr_wide = wide_rows(t.dR.p, t.dR.ld, t.M);
  p.r_wide = wide_rows(t.R.p, t.R.ld, t.M), p.h_wide = wide_rows(t.H.p, t.H.ld, t.M);
  p.dx_wide = wide_rows(t.dX.p, t.dX.ld, t.M), p.dh_wide = wide_rows(t.dH.p, t.dH.ld, t.M);
  p.gate_wide = wide_rows(t.gate.p, t.gate.ld, t.gates);
  p.vectors_wide = wide_rows(t.weight, 0, 1) && wide_rows(t.post_weight, 0, 1) && wide_rows(t.post_bias, 0, 1);
  const int rows = THREADS / p.threads;
  const int smem = rows * b.slots * words * kWord * 4;
  return ff::launch_early(stream, {dim3(static_cast<unsigned>(b.split.ctas)), rows * p.threads, 1, smem}, kern, p);
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
  cudaError_t e = t.N <= 4096 ? launch_rows<KIND, 512>(p, stream)
                  : t.N <= 8192
                      ? launch_rows<KIND, 1024>(p, stream)
                      : ff::launch_early(stream, {dim3(static_cast<unsigned>(p.split.ctas)), kWideThreads, 1, 0},
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
