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

No autograd history is recorded: ``linear`` and ``gated_linear`` refuse tensors that require grad
unless gradients are off (``torch.no_grad()``); the gradients are the backward functions' results.
"""
from __future__ import annotations

import ctypes

import torch

from . import binding
from .binding import T2S_OK, T2S_W_KN, T2S_W_NK, T2SError

ACTS = {"none": binding.T2S_ACT_NONE, "relu": binding.T2S_ACT_RELU, "silu": binding.T2S_ACT_SILU,
        "gelu": binding.T2S_ACT_GELU, "gelu_tanh": binding.T2S_ACT_GELU_TANH}
_SUFFIX = {torch.bfloat16: "_bf16", torch.float16: "_f16"}
_FUNCTIONS = {}
# A single token's call lasts a few microseconds on the device: what surrounds the launch is kept short.
_Tensor, _strided = torch.Tensor, torch.empty_strided
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
_grad_enabled = torch.is_grad_enabled
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)


def _function(name: str, dtype):
    """The C entry point of an operator for a type."""
    f = _FUNCTIONS.get((name, dtype))
    if f is None:
        full = name + _SUFFIX[dtype]
        f = binding.lib()[full]
        # Every argument is an integer in a register or stack slot of 64 bits, and ctypes converts
        # a c_void_p in two thirds of a c_int64's time.
        f.argtypes = [ctypes.c_void_p] * len(binding.SIGNATURES[full][0])
        f.restype = ctypes.c_int
        _FUNCTIONS[name, dtype] = f
    return f


def _first(t, name):
    """Type, device and its index of a call, set by its first tensor, and that tensor's pointer, row
    stride and sizes."""
    if not isinstance(t, _Tensor):
        raise TypeError("%s must be a bfloat16 or float16 CUDA tensor" % name)
    dtype, index = t.dtype, t.get_device()
    if dtype not in _SUFFIX or index < 0:
        raise TypeError("%s must be a bfloat16 or float16 CUDA tensor" % name)
    if index != _current_device():
        raise ValueError("%s must be on the current CUDA device" % name)
    size = t.shape
    if len(size) != 2:
        raise ValueError("%s must be 2-D" % name)
    rows, cols = size
    return dtype, t.device, index, t.data_ptr(), _row_stride(t, name, rows, cols), rows, cols


def _refuse_history(name):
    raise ValueError("%s records no autograd history, and an input requires grad: call it under torch.no_grad() and "
                     "%s_backward for the gradients" % (name, name))


def _refuse(t, name, dtype):
    if not isinstance(t, _Tensor) or t.dtype is not dtype or not t.is_cuda:
        raise TypeError("%s must be a %s CUDA tensor" % (name, dtype))
    raise ValueError("%s must be on the device of the other tensors" % name)


def _row_stride(t, name, rows, cols):
    ld, step = t.stride()
    if rows <= 1:  # its stride is never used: one that keeps the row in place
        ld = cols + 7 & -8
    if (step != 1 and cols > 1) or ld < cols:
        raise ValueError("%s must have contiguous rows that do not overlap" % name)
    return ld


def _matrix(t, name, dtype, index, shape):
    """Pointer and row stride of a matrix with contiguous rows."""
    if not isinstance(t, _Tensor) or t.dtype is not dtype or t.get_device() != index:
        _refuse(t, name, dtype)
    if t.shape != shape:
        raise ValueError("%s must be %d x %d, got %s" % (name, *shape, tuple(t.shape)))
    return t.data_ptr(), _row_stride(t, name, *shape)


def _inputs(t, name, dtype, index, rows):
    """Pointer, row stride and columns of a matrix of `rows` rows."""
    if not isinstance(t, _Tensor) or t.dtype is not dtype or t.get_device() != index:
        _refuse(t, name, dtype)
    size = t.shape
    if len(size) != 2 or size[0] != rows:
        raise ValueError("shape mismatch: %s %s for %d rows" % (name, tuple(size), rows))
    return t.data_ptr(), _row_stride(t, name, *size), size[1]


def _weight(t, name, dtype, index, k, n=None):
    """Pointer, row stride, order (T2S_W_KN or T2S_W_NK) and outputs of an inputs x outputs weight."""
    if not isinstance(t, _Tensor) or t.dtype is not dtype or t.get_device() != index:
        _refuse(t, name, dtype)
    size = t.shape
    if len(size) != 2:
        raise ValueError("%s must be 2-D" % name)
    if size[0] != k or (n is not None and size[1] != n):
        raise ValueError("shape mismatch: %s %s for %d inputs%s" % (
            name, tuple(size), k, "" if n is None else " and %d outputs" % n))
    n = size[1]
    a, b = t.stride()
    if b == 1 and (a >= n or k <= 1):
        return t.data_ptr(), a if k > 1 else n + 7 & -8, T2S_W_KN, n
    if a == 1 and (b >= k or n <= 1):
        return t.data_ptr(), b if n > 1 else k + 7 & -8, T2S_W_NK, n
    raise ValueError("%s must be row-major or the transpose of a row-major tensor" % name)


def _gradient(t, name, dtype, index, k, n, order):
    """Pointer and row stride of a weight's gradient, which has the weight's order."""
    if order == T2S_W_KN:
        return _matrix(t, name, dtype, index, (k, n))
    if not isinstance(t, _Tensor) or t.dim() != 2:
        raise ValueError("%s must be a 2-D tensor" % name)
    return _matrix(t.t(), name + ".t()", dtype, index, (n, k))


def _vector(t, name, dtype, index, n):
    if not isinstance(t, _Tensor) or t.dtype is not dtype or t.get_device() != index:
        _refuse(t, name, dtype)
    if t.shape != (n,) or (n > 1 and t.stride(0) != 1):
        raise ValueError("%s must be a contiguous vector of %d values" % (name, n))
    return t.data_ptr()


def _act(act):
    code = ACTS.get(act)
    if code is None:
        raise ValueError("act must be one of %s, got %r" % (", ".join(ACTS), act))
    return code


def _new(shape, strides, dtype, device, stream):
    """A tensor of the pool of the call's stream (None: the current one), so that the reuse of its
    memory is ordered there."""
    if stream is None:
        return _strided(shape, strides, dtype=dtype, device=device)
    with torch.cuda.stream(torch.cuda.ExternalStream(stream, device=device)):
        return _strided(shape, strides, dtype=dtype, device=device)


def _workspace(given, need, device, stream):
    """The workspace of a call (kept by the caller until it has been enqueued), its pointer and bytes."""
    if given is None:
        if not need:
            return None, None, 0
        given = _new((need,), (1,), torch.uint8, device, stream)
        return given, given.data_ptr(), need
    if not isinstance(given, _Tensor) or not given.is_cuda or not given.is_contiguous():
        raise TypeError("workspace must be a contiguous CUDA tensor")
    if given.get_device() != device.index:
        raise ValueError("workspace must be on the device of the other tensors")
    return given, given.data_ptr(), given.numel() * given.element_size()


def linear(x, w, bias=None, residual=None, act="none", out=None, preact=None, workspace=None, stream=None):
    """act(x @ w + bias) + residual; ``preact`` (a tensor of the output's shape) receives
    x @ w + bias, which ``linear_backward`` needs for an activation."""
    dtype, device, index, xp, ldx, M, K = _first(x, "x")
    wp, ldw, order, N = _weight(w, "w", dtype, index, K)
    bp = None if bias is None else _vector(bias, "bias", dtype, index, N)
    rp, ldr = (None, N) if residual is None else _matrix(residual, "residual", dtype, index, (M, N))
    zp, ldz = (None, N) if preact is None else _matrix(preact, "preact", dtype, index, (M, N))
    code = _act(act)
    if _grad_enabled() and (x.requires_grad or w.requires_grad or (bias is not None and bias.requires_grad)
                            or (residual is not None and residual.requires_grad)):
        _refuse_history("linear")
    if out is None:
        out = _new((M, N), (N, 1), dtype, device, stream)
        yp, ldy = out.data_ptr(), N
    else:
        yp, ldy = _matrix(out, "out", dtype, index, (M, N))
    # Rows that all start on 16-byte boundaries are read in place and need no workspace.
    need = binding.t2s_linear_workspace_size(M, N, K, 0) if (xp | wp | 2 * (ldx | ldw)) & 15 else 0
    keep, ws, size = _workspace(workspace, need, device, stream)
    f = _FUNCTIONS.get(("t2s_linear", dtype)) or _function("t2s_linear", dtype)
    rc = f(M, N, K, xp, ldx, wp, ldw, order, bp, rp, ldr, code, yp, ldy, zp, ldz, ws, size,
           _raw_stream(index) if stream is None else stream)
    if rc != T2S_OK:
        raise T2SError(rc, "t2s_linear" + _SUFFIX[dtype])
    return out


def linear_backward(dy, x, w, preact=None, act="none", dx=None, dw=None, db=False, workspace=None, stream=None):
    """(dx, dw, db) of ``linear``; the residual's gradient is dy itself. Each of dx, dw, db is
    None (allocated here), a tensor that receives it, or False (not computed). ``preact`` is
    what ``linear`` left there, needed for an ``act`` other than "none"."""
    dtype, device, index, yp, ldy, M, N = _first(dy, "dy")
    xp, ldx, K = _inputs(x, "x", dtype, index, M)
    wp, ldw, order, _ = _weight(w, "w", dtype, index, K, N)
    code = _act(act)
    zp, ldz = None, N
    if code != binding.T2S_ACT_NONE:
        if preact is None:
            raise ValueError("act %r needs the pre-activations" % act)
        zp, ldz = _matrix(preact, "preact", dtype, index, (M, N))
    dx, dxp, lddx = _output(dx, "dx", dtype, device, (M, K), stream)
    dw, dwp, lddw = _weight_output(dw, "dw", dtype, device, K, N, order, stream)
    if db is None:
        db = _new((N,), (1,), dtype, device, stream)
    dbp = None if db is False else _vector(db, "db", dtype, index, N)
    need = 0 if workspace is not None else binding.t2s_linear_backward_workspace_size(
        M, N, K, 0 if (xp | wp | yp | 2 * (ldx | ldw | ldy)) & 15 else 1)
    keep, ws, size = _workspace(workspace, need, device, stream)
    f = _FUNCTIONS.get(("t2s_linear_backward", dtype)) or _function("t2s_linear_backward", dtype)
    rc = f(M, N, K, yp, ldy, xp, ldx, wp, ldw, order, zp, ldz, code, dxp, lddx, dwp, lddw, dbp, ws, size,
           _raw_stream(index) if stream is None else stream)
    if rc != T2S_OK:
        raise T2SError(rc, "t2s_linear_backward" + _SUFFIX[dtype])
    return dx, dw, None if db is False else db


def _output(t, name, dtype, device, shape, stream):
    """An output, its pointer and row stride: given, allocated (None) or not wanted (False)."""
    if t is None:
        t = _new(shape, (shape[1], 1), dtype, device, stream)
        return t, t.data_ptr(), shape[1]
    if t is False:
        return None, None, shape[1]
    return (t, *_matrix(t, name, dtype, device.index, shape))


def _weight_output(t, name, dtype, device, k, n, order, stream):
    if t is None:
        kn = order == T2S_W_KN
        t = _new((k, n), (n, 1) if kn else (1, k), dtype, device, stream)
        return t, t.data_ptr(), n if kn else k
    if t is False:
        return None, None, max(k, n)
    return (t, *_gradient(t, name, dtype, device.index, k, n, order))


def gated_linear(x, w_gate, w_up, act="silu", out=None, preact=None, workspace=None, stream=None):
    """act(x @ w_gate) * (x @ w_up); ``preact``, a pair of tensors of the output's shape,
    receives x @ w_gate and x @ w_up, which ``gated_linear_backward`` needs."""
    dtype, device, index, xp, ldx, M, K = _first(x, "x")
    gp, ldg, order, N = _weight(w_gate, "w_gate", dtype, index, K)
    up, ldu, order_up, _ = _weight(w_up, "w_up", dtype, index, K, N)
    if order != order_up:
        raise ValueError("w_gate and w_up must have the same order")
    zg, ldzg, zu, ldzu = None, N, None, N
    if preact is not None:
        zg, ldzg = _matrix(preact[0], "preact[0]", dtype, index, (M, N))
        zu, ldzu = _matrix(preact[1], "preact[1]", dtype, index, (M, N))
    code = _act(act)
    if _grad_enabled() and (x.requires_grad or w_gate.requires_grad or w_up.requires_grad):
        _refuse_history("gated_linear")
    if out is None:
        out = _new((M, N), (N, 1), dtype, device, stream)
        hp, ldh = out.data_ptr(), N
    else:
        hp, ldh = _matrix(out, "out", dtype, index, (M, N))
    need = binding.t2s_gated_workspace_size(M, N, K, 0) if (xp | gp | up | 2 * (ldx | ldg | ldu)) & 15 else 0
    keep, ws, size = _workspace(workspace, need, device, stream)
    f = _FUNCTIONS.get(("t2s_gated", dtype)) or _function("t2s_gated", dtype)
    rc = f(M, N, K, xp, ldx, gp, ldg, up, ldu, order, code, hp, ldh, zg, ldzg, zu, ldzu, ws, size,
           _raw_stream(index) if stream is None else stream)
    if rc != T2S_OK:
        raise T2SError(rc, "t2s_gated" + _SUFFIX[dtype])
    return out


def gated_linear_backward(dh, x, w_gate, w_up, preact, act="silu", dx=None, dw_gate=None, dw_up=None,
                          workspace=None, stream=None):
    """(dx, dw_gate, dw_up) of ``gated_linear``; ``preact`` is the pair that it left there. Each
    output is None (allocated here), a tensor that receives it, or False (not computed)."""
    dtype, device, index, hp, ldh, M, N = _first(dh, "dh")
    xp, ldx, K = _inputs(x, "x", dtype, index, M)
    gp, ldg, order, _ = _weight(w_gate, "w_gate", dtype, index, K, N)
    up, ldu, order_up, _ = _weight(w_up, "w_up", dtype, index, K, N)
    if order != order_up:
        raise ValueError("w_gate and w_up must have the same order")
    zg, ldzg = _matrix(preact[0], "preact[0]", dtype, index, (M, N))
    zu, ldzu = _matrix(preact[1], "preact[1]", dtype, index, (M, N))
    code = _act(act)
    dx, dxp, lddx = _output(dx, "dx", dtype, device, (M, K), stream)
    dw_gate, dgp, lddg = _weight_output(dw_gate, "dw_gate", dtype, device, K, N, order, stream)
    dw_up, dup, lddu = _weight_output(dw_up, "dw_up", dtype, device, K, N, order, stream)
    need = 0 if workspace is not None else binding.t2s_gated_backward_workspace_size(
        M, N, K, 0 if (xp | gp | up | 2 * (ldx | ldg | ldu)) & 15 else 1)
    keep, ws, size = _workspace(workspace, need, device, stream)
    f = _FUNCTIONS.get(("t2s_gated_backward", dtype)) or _function("t2s_gated_backward", dtype)
    rc = f(M, N, K, hp, ldh, xp, ldx, gp, ldg, up, ldu, order, zg, ldzg, zu, ldzu, code, dxp, lddx, dgp, lddg, dup,
           lddu, ws, size, _raw_stream(index) if stream is None else stream)
    if rc != T2S_OK:
        raise T2SError(rc, "t2s_gated_backward" + _SUFFIX[dtype])
    return dx, dw_gate, dw_up
