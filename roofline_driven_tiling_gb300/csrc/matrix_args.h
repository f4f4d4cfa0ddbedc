// matrix_args.h -- argument checks shared by the C entry points that take strided matrices.
#pragma once

#include <cstdint>
#include <initializer_list>

#include "t2s_internal.h"

namespace t2s {

inline size_t up256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

inline bool bad_size(int64_t x) { return x < 0 || x > T2S_MAX_DIM; }

// A matrix argument of rows x cols values of `bytes` bytes (a vector: rows = 1).
struct Arg {
  const void* p;
  int64_t ld, rows, cols;
  unsigned bytes = 2;
};

inline bool bad_matrix(const Arg& a, bool required) {
  if (a.rows == 0 || a.cols == 0) return false;
  if (a.p == nullptr) return required;
  if ((reinterpret_cast<uintptr_t>(a.p) & (a.bytes - 1u)) != 0) return true;
  return a.ld < a.cols || a.ld > T2S_MAX_DIM;
}

inline bool same(const Arg& a, const Arg& b) {
  return a.p != nullptr && a.p == b.p && a.rows > 0 && a.cols > 0 && b.rows > 0 && b.cols > 0;
}

// Inputs that are required, inputs and outputs that may be absent, and no output that is
// another argument.
inline bool bad_arguments(std::initializer_list<Arg> required, std::initializer_list<Arg> optional,
                          std::initializer_list<Arg> outputs) {
  for (const Arg& a : required)
    if (bad_matrix(a, true)) return true;
  for (const Arg& a : optional)
    if (bad_matrix(a, false)) return true;
  for (const Arg* o = outputs.begin(); o != outputs.end(); ++o) {
    if (bad_matrix(*o, false)) return true;
    for (const Arg& a : required)
      if (same(*o, a)) return true;
    for (const Arg& a : optional)
      if (same(*o, a)) return true;
    for (const Arg* q = outputs.begin(); q != o; ++q)
      if (same(*o, *q)) return true;
  }
  return false;
}

inline int check_workspace(const void* p, size_t have, size_t need) {
  if (need == 0) return T2S_OK;
  if (p == nullptr || have < need || (reinterpret_cast<uintptr_t>(p) & 255u) != 0) return T2S_ERR_WORKSPACE;
  return T2S_OK;
}

// The return code of a call whose last CUDA call returned `e`.
inline int done(cudaError_t e) {
  if (e == cudaSuccess) return T2S_OK;
  set_last_cuda_error(e);
  return T2S_ERR_CUDA;
}

}  // namespace t2s
