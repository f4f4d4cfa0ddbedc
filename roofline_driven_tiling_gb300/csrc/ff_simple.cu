// ff_simple.cu -- the products of the feed-forward operators, one output per thread and k step,
// 32 x 32 tiles through shared memory: the definition for every size, layout and alignment.
#include <cuda_runtime.h>

#include <cstdint>
#include <type_traits>

#include "ff_internal.h"
#include "ff_math.cuh"

namespace t2s {
namespace ff {
namespace {

constexpr int kT = 32;

template <int KIND>
__device__ __forceinline__ float load(const Operand& o, int64_t i, int64_t k, int64_t extent, int64_t K) {
  if (i >= extent || k >= K) return 0.0f;
  return to_f32<KIND>(o.k_major ? o.p[i * o.ld + k] : o.p[k * o.ld + i]);
}

// 32 x 8 threads, four rows each.
template <int KIND>
__global__ void __launch_bounds__(256) ff_simple_kernel(const Task t) {
  __shared__ float sa[kT][kT + 1], sa2[kT][kT + 1], sb[kT][kT + 1], sb2[kT][kT + 1];
  const int tx = threadIdx.x, ty = threadIdx.y;
  const int64_t m0 = static_cast<int64_t>(blockIdx.y) * kT, n0 = static_cast<int64_t>(blockIdx.x) * kT;
  float s[4] = {}, s2[4] = {};
  for (int64_t k0 = 0; k0 < t.K; k0 += kT) {
    for (int i = ty; i < kT; i += 8) {
      sa[i][tx] = load<KIND>(t.A, m0 + i, k0 + tx, t.M, t.K);
      sb[i][tx] = load<KIND>(t.B, n0 + i, k0 + tx, t.N, t.K);
      if (t.form == kJoined) sa2[i][tx] = load<KIND>(t.A2, m0 + i, k0 + tx, t.M, t.K);
      if (t.form != kLinear) sb2[i][tx] = load<KIND>(t.B2, n0 + i, k0 + tx, t.N, t.K);
    }
    __syncthreads();
    for (int k = 0; k < kT; ++k)
      for (int r = 0; r < 4; ++r) {
        const int i = ty + 8 * r;
        s[r] = fmaf(sa[i][k], sb[tx][k], s[r]);
        if (t.form == kJoined) s[r] = fmaf(sa2[i][k], sb2[tx][k], s[r]);
        if (t.form == kGated) s2[r] = fmaf(sa[i][k], sb2[tx][k], s2[r]);
      }
    __syncthreads();
  }
  const int64_t n = n0 + tx;
  for (int r = 0; r < 4; ++r) {
    const int64_t m = m0 + ty + 8 * r;
    if (m >= t.M || n >= t.N) continue;
    float z = s[r];
    if (t.bias != nullptr) z += to_f32<KIND>(t.bias[n]);
    float y = 0.0f;
    with_act(t.act, [&](auto a) { y = act_value<decltype(a)::value>(z); });
    if (t.form == kGated) y *= s2[r];
    if (t.R.p != nullptr) y += to_f32<KIND>(t.R.p[m * t.R.ld + n]);
    if (t.Z.p != nullptr) t.Z.p[m * t.Z.ld + n] = from_f32<KIND>(z);
    if (t.Z2.p != nullptr) t.Z2.p[m * t.Z2.ld + n] = from_f32<KIND>(s2[r]);
    t.Y.p[m * t.Y.ld + n] = from_f32<KIND>(y);
  }
}

}  // namespace

cudaError_t run_simple(const Context& c, const Task& t) {
  // Row blocks along y (at most 65535 of them: larger M in several launches).
  for (int64_t m = 0; m < t.M; m += 65535 * kT) {
    Task part = t;
    part.M = t.M - m < 65535 * kT ? t.M - m : 65535 * kT;
    auto rows = [&](Operand& o) { if (o.p != nullptr) o.p += o.k_major ? m * o.ld : m; };
    rows(part.A);
    rows(part.A2);
    for (Matrix* x : {&part.R, &part.Y, &part.Z, &part.Z2})
      if (x->p != nullptr) x->p += m * x->ld;
    const dim3 grid(static_cast<unsigned>((part.N + kT - 1) / kT), static_cast<unsigned>((part.M + kT - 1) / kT));
    if (c.kind == kBf16)
      ff_simple_kernel<kBf16><<<grid, dim3(32, 8), 0, c.stream>>>(part);
    else
      ff_simple_kernel<kF16><<<grid, dim3(32, 8), 0, c.stream>>>(part);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace ff
}  // namespace t2s
