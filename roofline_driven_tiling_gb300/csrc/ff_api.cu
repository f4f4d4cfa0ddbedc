// ff_api.cu -- C entry points of the feed-forward operators: argument checks, workspace layout,
// and the kernels each operator takes.
#include <cuda_runtime.h>

#include <cstdint>
#include <initializer_list>

#include "ff_internal.h"
#include "t2s_internal.h"

namespace t2s {
namespace ff {
namespace {

size_t up256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }
int64_t up8(int64_t x) { return (x + 7) / 8 * 8; }
size_t plane_bytes(int64_t rows, int64_t cols) {
  return up256(static_cast<size_t>(rows) * static_cast<size_t>(up8(cols)) * 2);
}

bool bad_size(int64_t x) { return x < 0 || x > T2S_MAX_DIM; }

// A 16-bit matrix argument of rows x cols (a vector: rows = 1).
struct Arg {
  const void* p;
  int64_t ld, rows, cols;
};

bool bad_matrix(const Arg& a, bool required) {
  if (a.rows == 0 || a.cols == 0) return false;
  if (a.p == nullptr) return required;
  if ((reinterpret_cast<uintptr_t>(a.p) & 1u) != 0) return true;
  return a.ld < a.cols || a.ld > T2S_MAX_DIM;
}

bool same(const Arg& a, const Arg& b) {
  return a.p != nullptr && a.p == b.p && a.rows > 0 && a.cols > 0 && b.rows > 0 && b.cols > 0;
}

// Inputs that are required, inputs and outputs that may be absent, and no output that is
// another argument.
bool bad_arguments(std::initializer_list<Arg> required, std::initializer_list<Arg> optional,
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

bool bad_flags(int w_order, int act) {
  return (w_order != T2S_W_KN && w_order != T2S_W_NK) || act < T2S_ACT_NONE || act > T2S_ACT_GELU_TANH;
}

Arg weight_arg(const void* p, int64_t ld, int64_t K, int64_t N, int w_order) {
  return w_order == T2S_W_KN ? Arg{p, ld, K, N} : Arg{p, ld, N, K};
}

// The weight as the N x K operand of X W, and as the K x N operand of dZ W^T.
Operand weight_forward(const uint16_t* p, int64_t ld, int w_order) { return {p, ld, w_order == T2S_W_NK}; }
Operand weight_backward(const uint16_t* p, int64_t ld, int w_order) { return {p, ld, w_order == T2S_W_KN}; }

// Consecutive 256-byte aligned parts of the caller's workspace.
struct Workspace {
  uint8_t* p;
  size_t used = 0;
  void* take(size_t bytes) {
    void* at = p + used;
    used += up256(bytes);
    return at;
  }
};

// Whether the tensor cores' copies can read a matrix where it lies: all its rows on 16-byte
// boundaries (one row: only its start).
bool in_place(const void* p, int64_t rows, int64_t ld) { return aligned16(p, rows <= 1 ? 8 : ld); }

size_t copy_bytes(const void* p, int64_t rows, int64_t cols, int64_t ld) {
  return rows == 0 || cols == 0 || in_place(p, rows, ld) ? 0 : plane_bytes(rows, cols);
}

// The operands of a call that are copied into the workspace first, in one launch.
struct Copies {
  Workspace* ws;
  Copy list[kMaxCopies];
  int n = 0;

  // The rows x cols matrix `o` as it can be read: itself, or a copy.
  void read(int64_t rows, int64_t cols, Operand* o) {
    if (rows == 0 || cols == 0) return;
    if (in_place(o->p, rows, o->ld)) {
      if (rows <= 1) o->ld = up8(cols);
      return;
    }
    uint16_t* copy = static_cast<uint16_t*>(ws->take(plane_bytes(rows, cols)));
    list[n++] = {o->p, o->ld, rows, cols, copy};
    o->p = copy;
    o->ld = up8(cols);
  }
  void read_weight(int64_t K, int64_t N, int w_order, Operand* o) {
    if (w_order == T2S_W_KN) {
      read(K, N, o);
    } else {
      read(N, K, o);
    }
  }
};

size_t weight_copy_bytes(const void* p, int64_t K, int64_t N, int64_t ld, int w_order) {
  return w_order == T2S_W_KN ? copy_bytes(p, K, N, ld) : copy_bytes(p, N, K, ld);
}

int check_workspace(const void* p, size_t have, size_t need) {
  if (need == 0) return T2S_OK;
  if (p == nullptr || have < need || (reinterpret_cast<uintptr_t>(p) & 255u) != 0) return T2S_ERR_WORKSPACE;
  return T2S_OK;
}

int done(cudaError_t e) {
  if (e == cudaSuccess) return T2S_OK;
  set_last_cuda_error(e);
  return T2S_ERR_CUDA;
}

// The gradient of a weight: X^T D for a K x N weight, D^T X for an N x K one.
Task weight_gradient(int64_t M, int64_t N, int64_t K, Operand x, Operand d, int w_order, Matrix out) {
  Task t;
  x.k_major = d.k_major = false;
  t.M = w_order == T2S_W_KN ? K : N;
  t.N = w_order == T2S_W_KN ? N : K;
  t.K = M;
  t.A = w_order == T2S_W_KN ? x : d;
  t.B = w_order == T2S_W_KN ? d : x;
  t.Y = out;
  t.split = true;
  return t;
}

int linear(Kind kind, int64_t M, int64_t N, int64_t K, const uint16_t* X, int64_t ldx, const uint16_t* W,
           int64_t ldw, int w_order, const uint16_t* bias, const uint16_t* R, int64_t ldr, int act, uint16_t* Y,
           int64_t ldy, uint16_t* Z, int64_t ldz, void* workspace, size_t workspace_bytes, t2s_stream_t stream) {
  if (bad_size(M) || bad_size(N) || bad_size(K) || bad_flags(w_order, act)) return T2S_ERR_INVALID;
  const Arg x{X, ldx, M, K}, w = weight_arg(W, ldw, K, N, w_order), r{R, ldr, M, N}, y{Y, ldy, M, N};
  // Y may be R itself: every value of R is read by the thread block that then writes it.
  const bool in_place = R != nullptr && R == Y;
  if (in_place && ldr != ldy) return T2S_ERR_INVALID;
  if (bad_arguments({x, w}, {{bias, N, 1, N}, in_place ? Arg{nullptr, ldr, M, N} : r}, {y, {Z, ldz, M, N}}))
    return T2S_ERR_INVALID;
  if (M == 0 || N == 0) return T2S_OK;
  if (Y == nullptr) return T2S_ERR_INVALID;
  const int rc = check_workspace(workspace, workspace_bytes,
                                 copy_bytes(X, M, K, ldx) + weight_copy_bytes(W, K, N, ldw, w_order));
  if (rc != T2S_OK) return rc;
  Context c{kind, reinterpret_cast<cudaStream_t>(stream), nullptr};
  cudaError_t e = device_status_word(&c.status);
  if (e != cudaSuccess) return done(e);
  Task t;
  t.M = M, t.N = N, t.K = K;
  t.A = {X, ldx, true};
  t.B = weight_forward(W, ldw, w_order);
  t.bias = bias;
  t.R = {const_cast<uint16_t*>(R), ldr};
  t.act = act;
  t.Y = {Y, ldy};
  t.Z = {Z, ldz};
  Workspace ws{static_cast<uint8_t*>(workspace)};
  Copies copies{&ws};
  copies.read(M, K, &t.A);
  copies.read_weight(K, N, w_order, &t.B);
  if ((e = run_copies(c, copies.list, copies.n)) != cudaSuccess) return done(e);
  return done(run_products(c, &t, 1));
}

int linear_backward(Kind kind, int64_t M, int64_t N, int64_t K, const uint16_t* dY, int64_t lddy, const uint16_t* X,
                    int64_t ldx, const uint16_t* W, int64_t ldw, int w_order, const uint16_t* Z, int64_t ldz, int act,
                    uint16_t* dX, int64_t lddx, uint16_t* dW, int64_t lddw, uint16_t* db, void* workspace,
                    size_t workspace_bytes, t2s_stream_t stream) {
  if (bad_size(M) || bad_size(N) || bad_size(K) || bad_flags(w_order, act)) return T2S_ERR_INVALID;
  const Arg dy{dY, lddy, M, N}, z{Z, ldz, M, N};
  // X is only read for dW, W for dX, Z for an activation.
  const Arg x{dW != nullptr ? X : nullptr, ldx, M, K}, w = weight_arg(dX != nullptr ? W : nullptr, ldw, K, N, w_order);
  if (bad_arguments({dy}, {x, w, act != T2S_ACT_NONE ? z : Arg{nullptr, ldz, M, N}},
                    {{dX, lddx, M, K}, weight_arg(dW, lddw, K, N, w_order), {db, N, 1, N}}))
    return T2S_ERR_INVALID;
  if ((dW != nullptr && bad_matrix(x, N > 0)) || (dX != nullptr && bad_matrix(w, M > 0)) ||
      (act != T2S_ACT_NONE && bad_matrix(z, true)))
    return T2S_ERR_INVALID;
  const bool products = dX != nullptr || dW != nullptr;
  const bool plane = products && (act != T2S_ACT_NONE || !in_place(dY, M, lddy));
  const int64_t ldd = up8(N);
  const size_t sums = db != nullptr ? up256(db_partial_bytes(M, N)) : 0;
  const size_t pieces = dW != nullptr ? weight_partial_bytes(M, N, K, 1) : 0;
  const size_t need = (plane ? plane_bytes(M, N) : 0) + sums + pieces + (dW != nullptr ? copy_bytes(X, M, K, ldx) : 0) +
                      (dX != nullptr ? weight_copy_bytes(W, K, N, ldw, w_order) : 0);
  const int rc = check_workspace(workspace, workspace_bytes, need);
  if (rc != T2S_OK) return rc;
  Context c{kind, reinterpret_cast<cudaStream_t>(stream), nullptr};
  cudaError_t e = device_status_word(&c.status);
  if (e != cudaSuccess) return done(e);
  Workspace ws{static_cast<uint8_t*>(workspace)};
  Copies copies{&ws};
  if (pieces > 0) c.partials = static_cast<float*>(ws.take(c.partial_bytes = pieces));
  Operand d{dY, M <= 1 ? ldd : lddy, true};
  if (M > 0 && N > 0 && (plane || db != nullptr)) {
    uint16_t* dz = plane ? static_cast<uint16_t*>(ws.take(plane_bytes(M, N))) : nullptr;
    float* partials = sums > 0 ? static_cast<float*>(ws.take(sums)) : nullptr;
    e = run_act_backward(c, M, N, act, dY, lddy, Z, ldz, dz, ldd, db, partials);
    if (e != cudaSuccess) return done(e);
    if (plane) d = {dz, ldd, true};
  } else if (M == 0 && N > 0 && db != nullptr) {
    e = cudaMemsetAsync(db, 0, static_cast<size_t>(N) * 2, c.stream);
    if (e != cudaSuccess) return done(e);
  }
  Task tasks[2];
  int n = 0;
  if (dX != nullptr && M > 0 && K > 0) {
    Task& t = tasks[n++];
    t.M = M, t.N = K, t.K = N;
    t.A = d;
    t.B = weight_backward(W, ldw, w_order);
    t.Y = {dX, lddx};
    copies.read_weight(K, N, w_order, &t.B);
  }
  if (dW != nullptr && K > 0 && N > 0) {
    Operand x{X, ldx, false};
    copies.read(M, K, &x);
    tasks[n++] = weight_gradient(M, N, K, x, d, w_order, {dW, lddw});
  }
  if ((e = run_copies(c, copies.list, copies.n)) != cudaSuccess) return done(e);
  return done(run_products(c, tasks, n));
}

int gated(Kind kind, int64_t M, int64_t N, int64_t K, const uint16_t* X, int64_t ldx, const uint16_t* Wg,
          int64_t ldwg, const uint16_t* Wu, int64_t ldwu, int w_order, int act, uint16_t* H, int64_t ldh, uint16_t* G,
          int64_t ldg, uint16_t* U, int64_t ldu, void* workspace, size_t workspace_bytes, t2s_stream_t stream) {
  if (bad_size(M) || bad_size(N) || bad_size(K) || bad_flags(w_order, act)) return T2S_ERR_INVALID;
  if (bad_arguments({{X, ldx, M, K}, weight_arg(Wg, ldwg, K, N, w_order), weight_arg(Wu, ldwu, K, N, w_order)}, {},
                    {{H, ldh, M, N}, {G, ldg, M, N}, {U, ldu, M, N}}))
    return T2S_ERR_INVALID;
  if (M == 0 || N == 0) return T2S_OK;
  if (H == nullptr) return T2S_ERR_INVALID;
  const int rc = check_workspace(workspace, workspace_bytes,
                                 copy_bytes(X, M, K, ldx) + weight_copy_bytes(Wg, K, N, ldwg, w_order) +
                                     weight_copy_bytes(Wu, K, N, ldwu, w_order));
  if (rc != T2S_OK) return rc;
  Context c{kind, reinterpret_cast<cudaStream_t>(stream), nullptr};
  cudaError_t e = device_status_word(&c.status);
  if (e != cudaSuccess) return done(e);
  Task t;
  t.form = kGated;
  t.M = M, t.N = N, t.K = K;
  t.A = {X, ldx, true};
  t.B = weight_forward(Wg, ldwg, w_order);
  t.B2 = weight_forward(Wu, ldwu, w_order);
  t.act = act;
  t.Y = {H, ldh};
  t.Z = {G, ldg};
  t.Z2 = {U, ldu};
  Workspace ws{static_cast<uint8_t*>(workspace)};
  Copies copies{&ws};
  copies.read(M, K, &t.A);
  copies.read_weight(K, N, w_order, &t.B);
  copies.read_weight(K, N, w_order, &t.B2);
  if ((e = run_copies(c, copies.list, copies.n)) != cudaSuccess) return done(e);
  return done(run_products(c, &t, 1));
}

int gated_backward(Kind kind, int64_t M, int64_t N, int64_t K, const uint16_t* dH, int64_t lddh, const uint16_t* X,
                   int64_t ldx, const uint16_t* Wg, int64_t ldwg, const uint16_t* Wu, int64_t ldwu, int w_order,
                   const uint16_t* G, int64_t ldg, const uint16_t* U, int64_t ldu, int act, uint16_t* dX,
                   int64_t lddx, uint16_t* dWg, int64_t lddwg, uint16_t* dWu, int64_t lddwu, void* workspace,
                   size_t workspace_bytes, t2s_stream_t stream) {
  if (bad_size(M) || bad_size(N) || bad_size(K) || bad_flags(w_order, act)) return T2S_ERR_INVALID;
  // X is only read for the weights' gradients, the weights for dX.
  const bool dw = dWg != nullptr || dWu != nullptr;
  const Arg x{dw ? X : nullptr, ldx, M, K}, wg = weight_arg(dX ? Wg : nullptr, ldwg, K, N, w_order),
            wu = weight_arg(dX ? Wu : nullptr, ldwu, K, N, w_order);
  if (bad_arguments({{dH, lddh, M, N}, {G, ldg, M, N}, {U, ldu, M, N}}, {x, wg, wu},
                    {{dX, lddx, M, K}, weight_arg(dWg, lddwg, K, N, w_order), weight_arg(dWu, lddwu, K, N, w_order)}))
    return T2S_ERR_INVALID;
  if ((dw && bad_matrix(x, N > 0)) || (dX != nullptr && M > 0 && (bad_matrix(wg, true) || bad_matrix(wu, true))))
    return T2S_ERR_INVALID;
  const int64_t ldd = up8(N);
  size_t need = 2 * plane_bytes(M, N);
  const size_t pieces = dw ? weight_partial_bytes(M, N, K, (dWg != nullptr) + (dWu != nullptr)) : 0;
  need += pieces;
  if (dw) need += copy_bytes(X, M, K, ldx);
  if (dX != nullptr) need += weight_copy_bytes(Wg, K, N, ldwg, w_order) + weight_copy_bytes(Wu, K, N, ldwu, w_order);
  const int rc = check_workspace(workspace, workspace_bytes, need);
  if (rc != T2S_OK) return rc;
  Context c{kind, reinterpret_cast<cudaStream_t>(stream), nullptr};
  cudaError_t e = device_status_word(&c.status);
  if (e != cudaSuccess) return done(e);
  Workspace ws{static_cast<uint8_t*>(workspace)};
  Copies copies{&ws};
  if (pieces > 0) c.partials = static_cast<float*>(ws.take(c.partial_bytes = pieces));
  uint16_t *dG = nullptr, *dU = nullptr;
  if (M > 0 && N > 0 && (dw || dX != nullptr)) {
    dG = static_cast<uint16_t*>(ws.take(plane_bytes(M, N)));
    dU = static_cast<uint16_t*>(ws.take(plane_bytes(M, N)));
    e = run_gated_backward(c, M, N, act, dH, lddh, G, ldg, U, ldu, dG, dU, ldd);
    if (e != cudaSuccess) return done(e);
  }
  Task tasks[3];
  int n = 0;
  if (dX != nullptr && M > 0 && K > 0) {
    Task& t = tasks[n++];
    t.form = kJoined;
    t.M = M, t.N = K, t.K = N;
    t.A = {dG, ldd, true};
    t.A2 = {dU, ldd, true};
    t.B = weight_backward(Wg, ldwg, w_order);
    t.B2 = weight_backward(Wu, ldwu, w_order);
    t.Y = {dX, lddx};
    copies.read_weight(K, N, w_order, &t.B);
    copies.read_weight(K, N, w_order, &t.B2);
  }
  if (dw && K > 0 && N > 0) {
    Operand x{X, ldx, false};
    copies.read(M, K, &x);
    if (dWg != nullptr) tasks[n++] = weight_gradient(M, N, K, x, {dG, ldd, false}, w_order, {dWg, lddwg});
    if (dWu != nullptr) tasks[n++] = weight_gradient(M, N, K, x, {dU, ldd, false}, w_order, {dWu, lddwu});
  }
  if ((e = run_copies(c, copies.list, copies.n)) != cudaSuccess) return done(e);
  return done(run_products(c, tasks, n));
}

bool bad_sizes(int64_t M, int64_t N, int64_t K) { return bad_size(M) || bad_size(N) || bad_size(K); }

// X and a weight in either order as 16-byte aligned copies.
size_t copies_bytes(int64_t M, int64_t N, int64_t K, int weights) {
  const size_t kn = plane_bytes(K, N), nk = plane_bytes(N, K);
  return plane_bytes(M, K) + static_cast<size_t>(weights) * (kn > nk ? kn : nk);
}

}  // namespace
}  // namespace ff
}  // namespace t2s

using namespace t2s::ff;

extern "C" {

size_t t2s_linear_workspace_size(int64_t M, int64_t N, int64_t K, int aligned) {
  return bad_sizes(M, N, K) || aligned ? 0 : copies_bytes(M, N, K, 1);
}

size_t t2s_linear_backward_workspace_size(int64_t M, int64_t N, int64_t K, int aligned) {
  if (bad_sizes(M, N, K)) return 0;
  return plane_bytes(M, N) + up256(db_partial_bytes(M, N)) + weight_partial_bytes(M, N, K, 1) +
         (aligned ? 0 : copies_bytes(M, N, K, 1));
}

size_t t2s_gated_workspace_size(int64_t M, int64_t N, int64_t K, int aligned) {
  return bad_sizes(M, N, K) || aligned ? 0 : copies_bytes(M, N, K, 2);
}

size_t t2s_gated_backward_workspace_size(int64_t M, int64_t N, int64_t K, int aligned) {
  if (bad_sizes(M, N, K)) return 0;
  // The gradient of one weight can be split where those of two cannot.
  const size_t one = weight_partial_bytes(M, N, K, 1), two = weight_partial_bytes(M, N, K, 2);
  return 2 * plane_bytes(M, N) + (one > two ? one : two) + (aligned ? 0 : copies_bytes(M, N, K, 2));
}

int t2s_linear_bf16(int64_t M, int64_t N, int64_t K, const uint16_t* X, int64_t ldx, const uint16_t* W, int64_t ldw,
                    int w_order, const uint16_t* bias, const uint16_t* R, int64_t ldr, int act, uint16_t* Y,
                    int64_t ldy, uint16_t* Z, int64_t ldz, void* workspace, size_t workspace_bytes,
                    t2s_stream_t stream) {
  return linear(kBf16, M, N, K, X, ldx, W, ldw, w_order, bias, R, ldr, act, Y, ldy, Z, ldz, workspace,
                workspace_bytes, stream);
}

int t2s_linear_f16(int64_t M, int64_t N, int64_t K, const uint16_t* X, int64_t ldx, const uint16_t* W, int64_t ldw,
                   int w_order, const uint16_t* bias, const uint16_t* R, int64_t ldr, int act, uint16_t* Y,
                   int64_t ldy, uint16_t* Z, int64_t ldz, void* workspace, size_t workspace_bytes,
                   t2s_stream_t stream) {
  return linear(kF16, M, N, K, X, ldx, W, ldw, w_order, bias, R, ldr, act, Y, ldy, Z, ldz, workspace,
                workspace_bytes, stream);
}

int t2s_linear_backward_bf16(int64_t M, int64_t N, int64_t K, const uint16_t* dY, int64_t lddy, const uint16_t* X,
                             int64_t ldx, const uint16_t* W, int64_t ldw, int w_order, const uint16_t* Z, int64_t ldz,
                             int act, uint16_t* dX, int64_t lddx, uint16_t* dW, int64_t lddw, uint16_t* db,
                             void* workspace, size_t workspace_bytes, t2s_stream_t stream) {
  return linear_backward(kBf16, M, N, K, dY, lddy, X, ldx, W, ldw, w_order, Z, ldz, act, dX, lddx, dW, lddw, db,
                         workspace, workspace_bytes, stream);
}

int t2s_linear_backward_f16(int64_t M, int64_t N, int64_t K, const uint16_t* dY, int64_t lddy, const uint16_t* X,
                            int64_t ldx, const uint16_t* W, int64_t ldw, int w_order, const uint16_t* Z, int64_t ldz,
                            int act, uint16_t* dX, int64_t lddx, uint16_t* dW, int64_t lddw, uint16_t* db,
                            void* workspace, size_t workspace_bytes, t2s_stream_t stream) {
  return linear_backward(kF16, M, N, K, dY, lddy, X, ldx, W, ldw, w_order, Z, ldz, act, dX, lddx, dW, lddw, db,
                         workspace, workspace_bytes, stream);
}

int t2s_gated_bf16(int64_t M, int64_t N, int64_t K, const uint16_t* X, int64_t ldx, const uint16_t* Wg, int64_t ldwg,
                   const uint16_t* Wu, int64_t ldwu, int w_order, int act, uint16_t* H, int64_t ldh, uint16_t* G,
                   int64_t ldg, uint16_t* U, int64_t ldu, void* workspace, size_t workspace_bytes,
                   t2s_stream_t stream) {
  return gated(kBf16, M, N, K, X, ldx, Wg, ldwg, Wu, ldwu, w_order, act, H, ldh, G, ldg, U, ldu, workspace,
               workspace_bytes, stream);
}

int t2s_gated_f16(int64_t M, int64_t N, int64_t K, const uint16_t* X, int64_t ldx, const uint16_t* Wg, int64_t ldwg,
                  const uint16_t* Wu, int64_t ldwu, int w_order, int act, uint16_t* H, int64_t ldh, uint16_t* G,
                  int64_t ldg, uint16_t* U, int64_t ldu, void* workspace, size_t workspace_bytes,
                  t2s_stream_t stream) {
  return gated(kF16, M, N, K, X, ldx, Wg, ldwg, Wu, ldwu, w_order, act, H, ldh, G, ldg, U, ldu, workspace,
               workspace_bytes, stream);
}

int t2s_gated_backward_bf16(int64_t M, int64_t N, int64_t K, const uint16_t* dH, int64_t lddh, const uint16_t* X,
                            int64_t ldx, const uint16_t* Wg, int64_t ldwg, const uint16_t* Wu, int64_t ldwu,
                            int w_order, const uint16_t* G, int64_t ldg, const uint16_t* U, int64_t ldu, int act,
                            uint16_t* dX, int64_t lddx, uint16_t* dWg, int64_t lddwg, uint16_t* dWu, int64_t lddwu,
                            void* workspace, size_t workspace_bytes, t2s_stream_t stream) {
  return gated_backward(kBf16, M, N, K, dH, lddh, X, ldx, Wg, ldwg, Wu, ldwu, w_order, G, ldg, U, ldu, act, dX, lddx,
                        dWg, lddwg, dWu, lddwu, workspace, workspace_bytes, stream);
}

int t2s_gated_backward_f16(int64_t M, int64_t N, int64_t K, const uint16_t* dH, int64_t lddh, const uint16_t* X,
                           int64_t ldx, const uint16_t* Wg, int64_t ldwg, const uint16_t* Wu, int64_t ldwu,
                           int w_order, const uint16_t* G, int64_t ldg, const uint16_t* U, int64_t ldu, int act,
                           uint16_t* dX, int64_t lddx, uint16_t* dWg, int64_t lddwg, uint16_t* dWu, int64_t lddwu,
                           void* workspace, size_t workspace_bytes, t2s_stream_t stream) {
  return gated_backward(kF16, M, N, K, dH, lddh, X, ldx, Wg, ldwg, Wu, ldwu, w_order, G, ldg, U, ldu, act, dX, lddx,
                        dWg, lddwg, dWu, lddwu, workspace, workspace_bytes, stream);
}

}  // extern "C"
