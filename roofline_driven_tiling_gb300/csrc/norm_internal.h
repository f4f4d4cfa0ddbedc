// norm_internal.h -- norms with residual, gate and dropout, and dropout alone, between their C entry points
// (norm_api.cu) and the kernels.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "drop.cuh"
#include "ff_internal.h"
#include "t2s_internal.h"

namespace t2s {
namespace norm {

using ff::Kind;
using ff::Matrix;

struct Input {
  const uint16_t* p = nullptr;  // nullptr: absent
  int64_t ld = 0;
};

// What both directions take. Rows of `gate`: each for M / gates consecutive rows.
struct Shape {
  Kind kind;
  int64_t M, N;
  int norm, post;  // T2S_NORM_*
  float scale, eps;
  const uint16_t *weight, *bias, *post_weight, *post_bias;
  Input gate;
  int64_t gates;
  Dropout drop;
};

// r = scale X + gate drop(post(H)), y = norm(r). No H: r is X, and not written.
struct ForwardTask : Shape {
  Input X, H;
  Matrix R, Y;
};
cudaError_t run_forward(const ForwardTask& t, cudaStream_t stream);

// The gradients, from those of y (absent without a norm) and of r (absent where nothing else used r).
struct BackwardTask : Shape {
  Input dY, dR, R, H;
  Matrix dX, dH;
  uint16_t *dweight, *dbias, *dpost_weight, *dpost_bias;
  Matrix dgate;
  float* partials;  // backward_workspace_bytes
};
cudaError_t run_backward(const BackwardTask& t, cudaStream_t stream);
// For as many of the five vectors as are wanted (a gate counts with its rows).
size_t backward_workspace_bytes(int64_t M, int64_t N, int64_t gates, int vectors);

// Y = drop(X) + R.
struct DropoutTask {
  Kind kind;
  int64_t M, N;
  Input X, R;
  Dropout drop;
  Matrix Y;
};
cudaError_t run_dropout(const DropoutTask& t, cudaStream_t stream);

}  // namespace norm
}  // namespace t2s
