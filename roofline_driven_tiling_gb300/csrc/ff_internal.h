// ff_internal.h -- the feed-forward operators (linear, gated and their gradients) between their C
// entry points (ff_api.cu) and the kernels.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "t2s_internal.h"

namespace t2s {
namespace ff {

// 16-bit element types.
enum Kind : int { kBf16 = 1, kF16 = 0 };

// A product operand of `extent` x K values: `k_major` stores them as `extent` rows of K
// (contiguous along the sum), otherwise as K rows of `extent`. `ld` elements per row.
struct Operand {
  const uint16_t* p = nullptr;
  int64_t ld = 0;
  bool k_major = true;
};

struct Matrix {
  uint16_t* p = nullptr;  // nullptr: absent
  int64_t ld = 0;
};

// What follows a product's sums (one of the three forms).
enum Form : int {
  kLinear = 0,  // S = A B            Z = S + bias, Y = act(Z) + R
  kGated = 1,   // S = A B, S2 = A B2  Z = S, Z2 = S2, Y = act(S) * S2
  kJoined = 2,  // S = A B + A2 B2    Y = S
};

// One product M x N over K with its epilogue. B and B2 are N x K operands.
struct Task {
  Form form = kLinear;
  int64_t M = 0, N = 0, K = 0;
  Operand A, A2, B, B2;
  const uint16_t* bias = nullptr;
  Matrix R, Y, Z, Z2;
  int act = 0;
  bool split = false;  // its sum may be cut into pieces that Context::partials takes (no epilogue)
};

constexpr int kMaxProblems = 3;  // products of one launch

// Values of K that one accumulator sums. The tensor cores add in FP32 but truncate, always towards zero:
// a piece of this length loses at most 2^-13 of the sum of its magnitudes (measured with operands of one sign: 0.8 of
// that), a quarter of binary16's rounding. Longer sums are taken in pieces that are added in FP32.
constexpr int64_t kMaxPiece = 16384;

struct Context {
  Kind kind;
  cudaStream_t stream;
  unsigned* status;
  float* partials = nullptr;  // for weight gradients over many rows, see weight_partial_bytes
  size_t partial_bytes = 0;
};

inline bool aligned16(const void* p, int64_t ld) {
  return ((reinterpret_cast<uintptr_t>(p) | static_cast<uintptr_t>(ld * 2)) & 15u) == 0;
}

// How ff_pair.cu takes up to three products in one launch: sums per row of a tile, and pieces of the
// sum over K of those that may be split. `cost` is the expected time in microseconds.
struct PairPlan {
  int width = 256, splits = 1;
  double cost = 0.0;
};
PairPlan plan_pair(const Task* tasks, int n, int pairs, size_t partial_bytes);
// Up to three products in one launch (and one that adds the pieces), all of the gated form or none.
// Operands must be readable in place (aligned16), and rows of a single-row operand given a stride that is.
cudaError_t run_pair(const Context& c, const Task* tasks, const PairPlan& plan, int n);
// Bytes of Context::partials for the gradients of `weights` weights of K x N from M rows.
size_t weight_partial_bytes(int64_t M, int64_t N, int64_t K, int weights);

// How ff_rows.cu takes up to three products in one launch: CTAs along K, and for each product the
// rows of X per tile and the ring slots. `cost` is the expected time in microseconds.
struct RowsTile {
  int tm = 0, stages = 0;
  uint32_t stage_bytes = 0, tmem_cols = 0;
};
struct RowsPlan {
  int splits = 1, smem_bytes = 0;
  RowsTile tile[kMaxProblems];
  double cost = 0.0;
};
RowsPlan plan_rows(const Task* tasks, int n, int sms);
// Products with their sums split over clusters; operands as for run_pair.
cudaError_t run_rows(const Context& c, const Task* tasks, const RowsPlan& plan, int n);

// Up to three products, none or all of them of the gated form, each by the kernel that suits its sizes.
cudaError_t run_products(const Context& c, const Task* tasks, int n);

// dst = src, rows x cols, dst's rows padded to whole 16-byte words. Up to three copies in one launch.
struct Copy {
  const uint16_t* src;
  int64_t ld, rows, cols;
  uint16_t* dst;
};
constexpr int kMaxCopies = 3;
cudaError_t run_copies(const Context& c, const Copy* copies, int n);

// dZ = dY * act'(Z) (not stored if dZ is nullptr; Z is not read for act none) and, unless db is
// nullptr, its column sums.
cudaError_t run_act_backward(const Context& c, int64_t M, int64_t N, int act, const uint16_t* dY,
                             int64_t lddy, const uint16_t* Z, int64_t ldz, uint16_t* dZ,
                             int64_t lddz, uint16_t* db, float* partials);
// Bytes of `partials` that db needs for these sizes (0: it may be nullptr).
size_t db_partial_bytes(int64_t M, int64_t N);
// dG = dH * U * act'(G), dU = dH * act(G).
cudaError_t run_gated_backward(const Context& c, int64_t M, int64_t N, int act, const uint16_t* dH,
                               int64_t lddh, const uint16_t* G, int64_t ldg, const uint16_t* U,
                               int64_t ldu, uint16_t* dG, uint16_t* dU, int64_t ldd);

}  // namespace ff
}  // namespace t2s
