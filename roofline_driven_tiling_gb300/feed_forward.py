"""Feed-forward operators of a transformer block on bfloat16 or float16 CUDA tensors.

    linear           Z = x w + bias,  Y = act(Z) + residual
    linear_backward  dZ = dy * act'(Z),  dx = dZ w^T,  dw = x^T dZ,  db = dZ summed over rows
    gated_linear     G = x w_gate,  U = x w_up,  H = act(G) * U
    gated_linear_backward  dG = dh * U * act'(G),  dU = dh * act(G),
                           dx = dG w_gate^T + dU w_up^T,  dw_gate = x^T dG,  dw_up = x^T dU

Sums and activations are FP32; outputs have the inputs' type. Every matrix is 2-D with
contiguous rows and any row stride, so slices of larger tensors are taken as they are. A weight
is inputs x outputs, either row-major or the transpose of an outputs x inputs tensor
(``w.t()``); its gradient comes in the same order. Rows that start on 16-byte boundaries are
read in place, other operands are copied first: weights of odd width are best kept as a slice
of a tensor whose width is a multiple of 8.

``act`` is "none", "relu", "silu", "gelu" (erf) or "gelu_tanh". ``out`` may be the residual
itself. Outputs and workspaces that are not passed are allocated by torch. The work runs on
``stream`` (the integer value of a cudaStream_t; default: torch's current stream).
"""
from __future__ import annotations

import torch

from . import binding
from .binding import T2S_OK, T2S_W_KN, T2S_W_NK, T2SError

ACTS = {"none": binding.T2S_ACT_NONE, "relu": binding.T2S_ACT_RELU, "silu": binding.T2S_ACT_SILU,
        "gelu": binding.T2S_ACT_GELU, "gelu_tanh": binding.T2S_ACT_GELU_TANH}
_SUFFIX = {torch.bfloat16: "_bf16", torch.float16: "_f16"}
_FUNCTIONS = {}


def _function(name: str, dtype):
    """The C entry point of an operator for a type."""
    f = _FUNCTIONS.get((name, dtype))
    if f is None:
        f = _FUNCTIONS[name, dtype] = getattr(binding.lib(), name + _SUFFIX[dtype])
    return f


def _first(t, name):
    """Checks the tensor that sets the type and device of a call."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda or t.dtype not in _SUFFIX:
        raise TypeError("%s must be a bfloat16 or float16 CUDA tensor" % name)
    if t.get_device() != torch.cuda.current_device():
        raise ValueError("%s must be on the current CUDA device" % name)
    return t.dtype, t.get_device()


def _typed(t, name, like):
    if not isinstance(t, torch.Tensor) or not t.is_cuda or t.dtype != like.dtype:
        raise TypeError("%s must be a %s CUDA tensor" % (name, like.dtype))
    if t.get_device() != like.get_device():
        raise ValueError("%s must be on the device of the other tensors" % name)


def _rows(t, name, like, shape=None):
    """Pointer and row stride of a matrix with contiguous rows."""
    if t is not like:
        _typed(t, name, like)
    if t.dim() != 2:
        raise ValueError("%s must be 2-D" % name)
    rows, cols = t.shape
    if shape is not None and (rows, cols) != shape:
        raise ValueError("%s must be %d x %d, got %d x %d" % (name, *shape, rows, cols))
    ld, step = t.stride()
    if rows <= 1:  # its stride is never used: one that keeps the row in place
        ld = (cols + 7) // 8 * 8
    if (step != 1 and cols > 1) or ld < cols:
        raise ValueError("%s must have contiguous rows that do not overlap" % name)
    return t.data_ptr(), ld


def _weight(t, name, like, shape=None):
    """Pointer, row stride and order (T2S_W_KN or T2S_W_NK) of an inputs x outputs weight."""
    _typed(t, name, like)
    if t.dim() != 2:
        raise ValueError("%s must be 2-D" % name)
    k, n = t.shape
    if shape is not None and (k, n) != shape:
        raise ValueError("%s must be %d x %d, got %d x %d" % (name, *shape, k, n))
    a, b = t.stride()
    if b == 1 and (a >= n or k <= 1):
        return t.data_ptr(), a if k > 1 else (n + 7) // 8 * 8, T2S_W_KN
    if a == 1 and (b >= k or n <= 1):
        return t.data_ptr(), b if n > 1 else (k + 7) // 8 * 8, T2S_W_NK
    raise ValueError("%s must be row-major or the transpose of a row-major tensor" % name)


def _vector(t, name, like, n):
    _typed(t, name, like)
    if t.dim() != 1 or t.shape[0] != n or (n > 1 and t.stride(0) != 1):
        raise ValueError("%s must be a contiguous vector of %d values" % (name, n))
    return t.data_ptr()


def _act(act):
    if act not in ACTS:
        raise ValueError("act must be one of %s, got %r" % (", ".join(ACTS), act))
    return ACTS[act]


class _Call:
    """Where a call runs: its stream, and allocations that belong to that stream."""

    def __init__(self, device, stream):
        current = torch.cuda.current_stream(device).cuda_stream
        self.device, self.stream = device, current if stream is None else stream
        self.other = stream is not None and stream != current

    def empty(self, shape, dtype):
        if self.other:  # memory of that stream's pool, so that its reuse is ordered there
            with torch.cuda.stream(torch.cuda.ExternalStream(self.stream, device=self.device)):
                return torch.empty(shape, dtype=dtype, device=self.device)
        return torch.empty(shape, dtype=dtype, device=self.device)

    def workspace(self, given, need):
        """Pointer and size of the caller's workspace, or of a new one (kept by the third)."""
        if given is None:
            if not need:
                return None, 0, None
            given = self.empty(need, torch.uint8)
        elif not isinstance(given, torch.Tensor) or not given.is_cuda or not given.is_contiguous():
            raise TypeError("workspace must be a contiguous CUDA tensor")
        return given.data_ptr(), given.numel() * given.element_size(), given


def _in_place(*matrices) -> int:
    """1 if every (pointer, row stride) starts all its rows on 16-byte boundaries."""
    bits = 0
    for p, ld in matrices:
        bits |= p | 2 * ld
    return 0 if bits & 15 else 1


def _wanted(out, make):
    """An optional output: False is not wanted, None is allocated."""
    return None if out is False else make() if out is None else out


def linear(x, w, bias=None, residual=None, act="none", out=None, preact=None, workspace=None, stream=None):
    """act(x @ w + bias) + residual; ``preact`` (a tensor of the output's shape) receives
    x @ w + bias, which ``linear_backward`` needs for an activation."""
    dtype, device = _first(x, "x")
    xp, ldx = _rows(x, "x", x)
    M, K = x.shape
    wp, ldw, order = _weight(w, "w", x)
    if w.shape[0] != K:
        raise ValueError("shape mismatch: x %s, w %s" % (tuple(x.shape), tuple(w.shape)))
    N = w.shape[1]
    call = _Call(device, stream)
    bp = None if bias is None else _vector(bias, "bias", x, N)
    rp, ldr = (None, N) if residual is None else _rows(residual, "residual", x, (M, N))
    zp, ldz = (None, N) if preact is None else _rows(preact, "preact", x, (M, N))
    if out is None:
        out, ldy = call.empty((M, N), dtype), N
        yp = out.data_ptr()
    else:
        yp, ldy = _rows(out, "out", x, (M, N))
    need = 0 if _in_place((xp, ldx), (wp, ldw)) else binding.lib().t2s_linear_workspace_size(M, N, K, 0)
    ws, size, keep = call.workspace(workspace, need)
    rc = _function("t2s_linear", dtype)(M, N, K, xp, ldx, wp, ldw, order, bp, rp, ldr, _act(act), yp, ldy, zp, ldz,
                                        ws, size, call.stream)
    if rc != T2S_OK:
        raise T2SError(rc, "t2s_linear" + _SUFFIX[dtype])
    return out


def linear_backward(dy, x, w, preact=None, act="none", dx=None, dw=None, db=False, workspace=None, stream=None):
    """(dx, dw, db) of ``linear``; the residual's gradient is dy itself. Each of dx, dw, db is
    None (allocated here), a tensor that receives it, or False (not computed). ``preact`` is
    what ``linear`` left there, needed for an ``act`` other than "none"."""
    dtype, device = _first(dy, "dy")
    yp, ldy = _rows(dy, "dy", dy)
    M, N = dy.shape
    xp, ldx = _rows(x, "x", dy)
    K = x.shape[1]
    if x.shape[0] != M:
        raise ValueError("shape mismatch: dy %s, x %s" % (tuple(dy.shape), tuple(x.shape)))
    wp, ldw, order = _weight(w, "w", dy, (K, N))
    code = _act(act)
    if code != binding.T2S_ACT_NONE and preact is None:
        raise ValueError("act %r needs the pre-activations" % act)
    zp, ldz = (None, N) if preact is None or code == binding.T2S_ACT_NONE else _rows(preact, "preact", dy, (M, N))
    call = _Call(device, stream)
    dx = _wanted(dx, lambda: call.empty((M, K), dtype))
    dw = _wanted(dw, lambda: call.empty((K, N), dtype) if order == T2S_W_KN else call.empty((N, K), dtype).t())
    db = _wanted(db, lambda: call.empty((N,), dtype))
    dxp, lddx = (None, K) if dx is None else _rows(dx, "dx", dy, (M, K))
    dwp, lddw = (None, max(K, N)) if dw is None else _gradient(dw, "dw", dy, (K, N), order)
    dbp = None if db is None else _vector(db, "db", dy, N)
    need = binding.lib().t2s_linear_backward_workspace_size(M, N, K, _in_place((xp, ldx), (wp, ldw), (yp, ldy)))
    ws, size, keep = call.workspace(workspace, need)
    rc = _function("t2s_linear_backward", dtype)(M, N, K, yp, ldy, xp, ldx, wp, ldw, order, zp, ldz, code, dxp, lddx,
                                                 dwp, lddw, dbp, ws, size, call.stream)
    if rc != T2S_OK:
        raise T2SError(rc, "t2s_linear_backward" + _SUFFIX[dtype])
    return dx, dw, db


def _gradient(t, name, like, shape, order):
    """Pointer and row stride of a weight's gradient, which has the weight's order."""
    if order == T2S_W_KN:
        return _rows(t, name, like, shape)
    _typed(t, name, like)
    if t.dim() != 2:
        raise ValueError("%s must be 2-D" % name)
    return _rows(t.t(), name + ".t()", like, (shape[1], shape[0]))


def gated_linear(x, w_gate, w_up, act="silu", out=None, preact=None, workspace=None, stream=None):
    """act(x @ w_gate) * (x @ w_up); ``preact``, a pair of tensors of the output's shape,
    receives x @ w_gate and x @ w_up, which ``gated_linear_backward`` needs."""
    dtype, device = _first(x, "x")
    xp, ldx = _rows(x, "x", x)
    M, K = x.shape
    gp, ldg, order = _weight(w_gate, "w_gate", x)
    if w_gate.shape[0] != K:
        raise ValueError("shape mismatch: x %s, w_gate %s" % (tuple(x.shape), tuple(w_gate.shape)))
    N = w_gate.shape[1]
    up, ldu, order_up = _weight(w_up, "w_up", x, (K, N))
    if order != order_up:
        raise ValueError("w_gate and w_up must have the same order")
    call = _Call(device, stream)
    if out is None:
        out, ldh = call.empty((M, N), dtype), N
        hp = out.data_ptr()
    else:
        hp, ldh = _rows(out, "out", x, (M, N))
    zg, ldzg, zu, ldzu = None, N, None, N
    if preact is not None:
        zg, ldzg = _rows(preact[0], "preact[0]", x, (M, N))
        zu, ldzu = _rows(preact[1], "preact[1]", x, (M, N))
    need = 0
    if not _in_place((xp, ldx), (gp, ldg), (up, ldu)):
        need = binding.lib().t2s_gated_workspace_size(M, N, K, 0)
    ws, size, keep = call.workspace(workspace, need)
    rc = _function("t2s_gated", dtype)(M, N, K, xp, ldx, gp, ldg, up, ldu, order, _act(act), hp, ldh, zg, ldzg, zu,
                                       ldzu, ws, size, call.stream)
    if rc != T2S_OK:
        raise T2SError(rc, "t2s_gated" + _SUFFIX[dtype])
    return out


def gated_linear_backward(dh, x, w_gate, w_up, preact, act="silu", dx=None, dw_gate=None, dw_up=None,
                          workspace=None, stream=None):
    """(dx, dw_gate, dw_up) of ``gated_linear``; ``preact`` is the pair that it left there. Each
    output is None (allocated here), a tensor that receives it, or False (not computed)."""
    dtype, device = _first(dh, "dh")
    hp, ldh = _rows(dh, "dh", dh)
    M, N = dh.shape
    xp, ldx = _rows(x, "x", dh)
    K = x.shape[1]
    if x.shape[0] != M:
        raise ValueError("shape mismatch: dh %s, x %s" % (tuple(dh.shape), tuple(x.shape)))
    gp, ldg, order = _weight(w_gate, "w_gate", dh, (K, N))
    up, ldu, order_up = _weight(w_up, "w_up", dh, (K, N))
    if order != order_up:
        raise ValueError("w_gate and w_up must have the same order")
    zg, ldzg = _rows(preact[0], "preact[0]", dh, (M, N))
    zu, ldzu = _rows(preact[1], "preact[1]", dh, (M, N))
    call = _Call(device, stream)

    def weight_like():
        return call.empty((K, N), dtype) if order == T2S_W_KN else call.empty((N, K), dtype).t()

    dx = _wanted(dx, lambda: call.empty((M, K), dtype))
    dw_gate, dw_up = _wanted(dw_gate, weight_like), _wanted(dw_up, weight_like)
    dxp, lddx = (None, K) if dx is None else _rows(dx, "dx", dh, (M, K))
    dgp, lddg = (None, max(K, N)) if dw_gate is None else _gradient(dw_gate, "dw_gate", dh, (K, N), order)
    dup, lddu = (None, max(K, N)) if dw_up is None else _gradient(dw_up, "dw_up", dh, (K, N), order)
    need = binding.lib().t2s_gated_backward_workspace_size(M, N, K, _in_place((xp, ldx), (gp, ldg), (up, ldu)))
    ws, size, keep = call.workspace(workspace, need)
    rc = _function("t2s_gated_backward", dtype)(M, N, K, hp, ldh, xp, ldx, gp, ldg, up, ldu, order, zg, ldzg, zu, ldzu,
                                                _act(act), dxp, lddx, dgp, lddg, dup, lddu, ws, size, call.stream)
    if rc != T2S_OK:
        raise T2SError(rc, "t2s_gated_backward" + _SUFFIX[dtype])
    return dx, dw_gate, dw_up
