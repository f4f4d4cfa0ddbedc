// norm_api.cu -- C entry points of the norms with residual, gate and dropout, their gradients, and dropout
// alone: argument checks and the empty cases.
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "matrix_args.h"
#include "norm_internal.h"

namespace t2s {
namespace norm {
namespace {

bool bad_norm(int n) { return n < T2S_NORM_NONE || n > T2S_NORM_LAYER; }

bool bad_drop(int dropped, const int64_t* seed_device) {
  return dropped < 0 || dropped > 65536 || (reinterpret_cast<uintptr_t>(seed_device) & 7u) != 0;
}

Dropout drop_of(int dropped, const int64_t* seed_device, int64_t seed, int64_t sequence) {
  Dropout d;
  d.seed_at = seed_device;
  d.seed = static_cast<uint64_t>(seed);
  d.sequence = static_cast<uint64_t>(sequence);
  d.dropped = static_cast<uint32_t>(dropped);
  d.factor = dropped < 65536 ? 65536.0f / static_cast<float>(65536 - dropped) : 0.0f;
  return d;
}

bool bad_shape(int64_t M, int64_t N, int norm, int post, int64_t gates, float scale, float eps) {
  return bad_size(M) || bad_size(N) || bad_norm(norm) || bad_norm(post) || gates < 1 || M % gates != 0 ||
         !std::isfinite(scale) || !std::isfinite(eps) || eps < 0.0f;
}

int forward(Kind kind, int64_t M, int64_t N, int norm, int post, const uint16_t* X, int64_t ldx, const uint16_t* H,
            int64_t ldh, const uint16_t* weight, const uint16_t* bias, const uint16_t* post_weight,
            const uint16_t* post_bias, const uint16_t* gate, int64_t ldgate, int64_t gates, float scale, float eps,
            int dropped, const int64_t* seed_device, int64_t seed, int64_t sequence, uint16_t* R, int64_t ldr,
            uint16_t* Y, int64_t ldy, t2s_stream_t stream) {
  if (bad_shape(M, N, norm, post, gates, scale, eps) || bad_drop(dropped, seed_device)) return T2S_ERR_INVALID;
  if (norm == T2S_NORM_NONE && (weight != nullptr || bias != nullptr || Y != nullptr)) return T2S_ERR_INVALID;
  if (post == T2S_NORM_NONE && (post_weight != nullptr || post_bias != nullptr)) return T2S_ERR_INVALID;
  if (H == nullptr && M > 0 && N > 0 &&
      (post != T2S_NORM_NONE || gate != nullptr || dropped != 0 || scale != 1.0f || R != nullptr))
    return T2S_ERR_INVALID;
  // R may be X itself: every value of X is read by the thread that then writes it.
  const bool in_place = R != nullptr && R == X;
  if (in_place && ldr != ldx && M > 1) return T2S_ERR_INVALID;
  const Arg x{X, ldx, M, N}, r{in_place ? nullptr : R, ldr, M, N}, g{gate, ldgate, gates, N};
  if (bad_arguments({x}, {{H, ldh, M, N}, {weight, N, 1, N}, {bias, N, 1, N}, {post_weight, N, 1, N},
                          {post_bias, N, 1, N}, g}, {r, {Y, ldy, M, N}}))
    return T2S_ERR_INVALID;
  if (in_place && (ldr < N || ldr > T2S_MAX_DIM || same({R, ldr, M, N}, {H, ldh, M, N}) || same({R, ldr, M, N}, g)))
    return T2S_ERR_INVALID;
  if (M == 0 || N == 0) return T2S_OK;
  if ((H != nullptr && R == nullptr) || (norm != T2S_NORM_NONE && Y == nullptr) ||
      (H == nullptr && norm == T2S_NORM_NONE))
    return T2S_ERR_INVALID;
  ForwardTask t;
  t.kind = kind, t.M = M, t.N = N, t.norm = norm, t.post = post, t.scale = scale, t.eps = eps;
  t.weight = weight, t.bias = bias, t.post_weight = post_weight, t.post_bias = post_bias;
  t.gate = {gate, ldgate}, t.gates = gates;
  t.drop = drop_of(dropped, seed_device, seed, sequence);
  t.X = {X, ldx}, t.H = {H, ldh}, t.R = {R, ldr}, t.Y = {Y, ldy};
  return done(run_forward(t, reinterpret_cast<cudaStream_t>(stream)));
}

// Zeros in a gradient that is a sum over no rows.
cudaError_t clear(uint16_t* p, int64_t ld, int64_t rows, int64_t cols, cudaStream_t stream) {
  if (p == nullptr || rows == 0) return cudaSuccess;
  const size_t width = static_cast<size_t>(cols) * 2;
  return rows == 1 ? cudaMemsetAsync(p, 0, width, stream)
                   : cudaMemset2DAsync(p, static_cast<size_t>(ld) * 2, 0, width, static_cast<size_t>(rows), stream);
}

int backward(Kind kind, int64_t M, int64_t N, int norm, int post, const uint16_t* dY, int64_t lddy, const uint16_t* dR,
             int64_t lddr, const uint16_t* R, int64_t ldr, const uint16_t* H, int64_t ldh, const uint16_t* weight,
             const uint16_t* post_weight, const uint16_t* post_bias, const uint16_t* gate, int64_t ldgate,
             int64_t gates, float scale, float eps, int dropped, const int64_t* seed_device, int64_t seed,
             int64_t sequence, uint16_t* dX, int64_t lddx, uint16_t* dH, int64_t lddh, uint16_t* dweight,
             uint16_t* dbias, uint16_t* dpost_weight, uint16_t* dpost_bias, uint16_t* dgate, int64_t lddgate,
             void* workspace, size_t workspace_bytes, t2s_stream_t stream) {
  if (bad_shape(M, N, norm, post, gates, scale, eps) || bad_drop(dropped, seed_device)) return T2S_ERR_INVALID;
  if (norm == T2S_NORM_NONE && (weight != nullptr || dY != nullptr || dweight != nullptr || dbias != nullptr))
    return T2S_ERR_INVALID;
  if (post == T2S_NORM_NONE &&
      (post_weight != nullptr || post_bias != nullptr || dpost_weight != nullptr || dpost_bias != nullptr))
    return T2S_ERR_INVALID;
  if (H == nullptr && M > 0 && N > 0 &&
      (post != T2S_NORM_NONE || gate != nullptr || dropped != 0 || dH != nullptr || dgate != nullptr || scale != 1.0f))
    return T2S_ERR_INVALID;
  const Arg dy{dY, lddy, M, N}, r{norm != T2S_NORM_NONE ? R : nullptr, ldr, M, N};
  if (bad_arguments({}, {dy, {dR, lddr, M, N}, r, {H, ldh, M, N}, {weight, N, 1, N}, {post_weight, N, 1, N},
                         {post_bias, N, 1, N}, {gate, ldgate, gates, N}},
                    {{dX, lddx, M, N}, {dH, lddh, M, N}, {dweight, N, 1, N}, {dbias, N, 1, N}, {dpost_weight, N, 1, N},
                     {dpost_bias, N, 1, N}, {dgate, lddgate, gates, N}}))
    return T2S_ERR_INVALID;
  if (norm != T2S_NORM_NONE && (bad_matrix(dy, true) || bad_matrix(r, true))) return T2S_ERR_INVALID;
  if (N == 0) return T2S_OK;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (M == 0) {
    cudaError_t e = cudaSuccess;
    for (uint16_t* p : {dweight, dbias, dpost_weight, dpost_bias})
      if (e == cudaSuccess) e = clear(p, N, 1, N, s);
    if (e == cudaSuccess) e = clear(dgate, lddgate, gates, N, s);
    return done(e);
  }
  const int vectors = (dweight != nullptr) + (dbias != nullptr) + (dpost_weight != nullptr) + (dpost_bias != nullptr) +
                      (dgate != nullptr);
  const int rc = check_workspace(workspace, workspace_bytes, backward_workspace_bytes(M, N, gates, vectors));
  if (rc != T2S_OK) return rc;
  BackwardTask t;
  t.kind = kind, t.M = M, t.N = N, t.norm = norm, t.post = post, t.scale = scale, t.eps = eps;
  t.weight = weight, t.bias = nullptr, t.post_weight = post_weight, t.post_bias = post_bias;
  t.gate = {gate, ldgate}, t.gates = gates;
  t.drop = drop_of(dropped, seed_device, seed, sequence);
  t.dY = {dY, lddy}, t.dR = {dR, lddr}, t.R = {R, ldr}, t.H = {H, ldh}, t.dX = {dX, lddx}, t.dH = {dH, lddh};
  t.dweight = dweight, t.dbias = dbias, t.dpost_weight = dpost_weight, t.dpost_bias = dpost_bias;
  t.dgate = {dgate, lddgate};
  t.partials = static_cast<float*>(workspace);
  return done(run_backward(t, s));
}

int dropout(Kind kind, int64_t M, int64_t N, const uint16_t* X, int64_t ldx, const uint16_t* R, int64_t ldr,
            int dropped, const int64_t* seed_device, int64_t seed, int64_t sequence, uint16_t* Y, int64_t ldy,
            t2s_stream_t stream) {
  if (bad_size(M) || bad_size(N) || bad_drop(dropped, seed_device)) return T2S_ERR_INVALID;
  if (bad_matrix({X, ldx, M, N}, true) || bad_matrix({R, ldr, M, N}, false) || bad_matrix({Y, ldy, M, N}, true))
    return T2S_ERR_INVALID;
  // Y may be one of the inputs: every value is read by the thread that then writes it.
  if (M > 1 && N > 0 && ((Y == X && ldy != ldx) || (Y == R && ldy != ldr))) return T2S_ERR_INVALID;
  if (M == 0 || N == 0) return T2S_OK;
  DropoutTask t;
  t.kind = kind, t.M = M, t.N = N;
  t.X = {X, ldx}, t.R = {R, ldr}, t.Y = {Y, ldy};
  t.drop = drop_of(dropped, seed_device, seed, sequence);
  return done(run_dropout(t, reinterpret_cast<cudaStream_t>(stream)));
}

}  // namespace
}  // namespace norm
}  // namespace t2s

using namespace t2s::norm;
using t2s::ff::kBf16;
using t2s::ff::kF16;

extern "C" {

size_t t2s_residual_norm_backward_workspace_size(int64_t M, int64_t N, int64_t gates, int vectors) {
  if (t2s::bad_size(M) || t2s::bad_size(N) || gates < 1 || M % gates != 0 || vectors < 0 || vectors > 5) return 0;
  return t2s::up256(backward_workspace_bytes(M, N, gates, vectors));
}

#define T2S_RESIDUAL_NORM(SUFFIX, KIND)                                                                               \
  int t2s_residual_norm_##SUFFIX(int64_t M, int64_t N, int norm, int post, const uint16_t* X, int64_t ldx,            \
                                 const uint16_t* H, int64_t ldh, const uint16_t* weight, const uint16_t* bias,        \
                                 const uint16_t* post_weight, const uint16_t* post_bias, const uint16_t* gate,        \
                                 int64_t ldgate, int64_t gates, float scale, float eps, int dropped_of_65536,         \
                                 const int64_t* seed_device, int64_t seed, int64_t sequence, uint16_t* R,             \
                                 int64_t ldr, uint16_t* Y, int64_t ldy, t2s_stream_t stream) {                        \
    return forward(KIND, M, N, norm, post, X, ldx, H, ldh, weight, bias, post_weight, post_bias, gate, ldgate, gates, \
                   scale, eps, dropped_of_65536, seed_device, seed, sequence, R, ldr, Y, ldy, stream);                \
  }                                                                                                                   \
  int t2s_residual_norm_backward_##SUFFIX(                                                                            \
      int64_t M, int64_t N, int norm, int post, const uint16_t* dY, int64_t lddy, const uint16_t* dR, int64_t lddr,   \
      const uint16_t* R, int64_t ldr, const uint16_t* H, int64_t ldh, const uint16_t* weight,                         \
      const uint16_t* post_weight, const uint16_t* post_bias, const uint16_t* gate, int64_t ldgate, int64_t gates,    \
      float scale, float eps, int dropped_of_65536, const int64_t* seed_device, int64_t seed, int64_t sequence,       \
      uint16_t* dX, int64_t lddx, uint16_t* dH, int64_t lddh, uint16_t* dweight, uint16_t* dbias,                     \
      uint16_t* dpost_weight, uint16_t* dpost_bias, uint16_t* dgate, int64_t lddgate, void* workspace,                \
      size_t workspace_bytes, t2s_stream_t stream) {                                                                  \
    return backward(KIND, M, N, norm, post, dY, lddy, dR, lddr, R, ldr, H, ldh, weight, post_weight, post_bias, gate, \
                    ldgate, gates, scale, eps, dropped_of_65536, seed_device, seed, sequence, dX, lddx, dH, lddh,     \
                    dweight, dbias, dpost_weight, dpost_bias, dgate, lddgate, workspace, workspace_bytes, stream);    \
  }                                                                                                                   \
  int t2s_dropout_##SUFFIX(int64_t M, int64_t N, const uint16_t* X, int64_t ldx, const uint16_t* R, int64_t ldr,      \
                           int dropped_of_65536, const int64_t* seed_device, int64_t seed, int64_t sequence,          \
                           uint16_t* Y, int64_t ldy, t2s_stream_t stream) {                                           \
    return dropout(KIND, M, N, X, ldx, R, ldr, dropped_of_65536, seed_device, seed, sequence, Y, ldy, stream);        \
  }

T2S_RESIDUAL_NORM(bf16, kBf16)
T2S_RESIDUAL_NORM(f16, kF16)

}  // extern "C"
