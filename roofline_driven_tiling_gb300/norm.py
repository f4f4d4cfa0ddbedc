"""What stands between two blocks of a transformer, on bfloat16 or float16 CUDA tensors.

    residual_norm            n = post_norm(h) * post_weight + post_bias
                             r = scale * x + gate * dropout(n),  y = norm(r) * weight + bias
    residual_norm_backward   its gradients
    dropout                  x with values dropped, plus a residual
    dropout_backward         its gradient

Norms are "rms" (v / sqrt(mean(v^2) + eps)), "layer" ((v - mean) / sqrt(variance + eps)) or "none",
each over a row. Statistics and sums are FP32; r is rounded to the inputs' type, y is the norm of the
rounded r; outputs have the inputs' type. Every matrix is 2-D with contiguous rows and any row
stride. A gate is a vector (a value for each channel), or a matrix whose rows serve equal numbers of
consecutive rows of x (a gate for each sample of a batch).

Dropout keeps no mask: a value's fate depends on ``seed``, ``sequence`` and its place alone. Give
every call of a training step its own ``sequence`` and every step its own ``seed``, and the backward
pass those of its forward pass. ``p`` is rounded to a multiple of 2^-16; kept values are divided by
the probability of staying. ``seed`` is a number or a one-element int64 tensor on the device, which
the kernels read when they run: a captured graph draws anew when the tensor has changed.

The work runs on ``stream`` (the integer value of a cudaStream_t; default: torch's current stream).
No autograd history is recorded: the forward functions refuse tensors that require grad unless
gradients are off (``torch.no_grad()``); the gradients are the backward functions' results.
"""
from __future__ import annotations

import ctypes
from typing import NamedTuple

import torch

from . import binding
from .binding import T2S_OK, T2SError
from .feed_forward import (_first, _grad_enabled, _matrix, _new, _output, _raw_stream, _refuse_history,
                           _SUFFIX, _Tensor, _vector, _workspace)

NORMS = {"none": binding.T2S_NORM_NONE, "rms": binding.T2S_NORM_RMS, "layer": binding.T2S_NORM_LAYER}
_FUNCTIONS = {}


class ResidualNormGradients(NamedTuple):
    """The gradients of ``residual_norm``'s inputs; None for inputs that were absent or not wanted."""
    dx: object
    dh: object
    dweight: object
    dbias: object
    dgate: object
    dpost_weight: object
    dpost_bias: object


def _function(name, dtype):
    f = _FUNCTIONS.get((name, dtype))
    if f is None:
        full = name + _SUFFIX[dtype]
        f = binding.lib()[full]
        # All arguments but the two floats are integers, which convert quickest as pointers.
        f.argtypes = [t if t is ctypes.c_float else ctypes.c_void_p for t in binding.SIGNATURES[full][0]]
        f.restype = ctypes.c_int
        _FUNCTIONS[name, dtype] = f
    return f


_workspace_size = None


def _function_of_size():
    global _workspace_size
    _workspace_size = binding.lib().t2s_residual_norm_backward_workspace_size
    return _workspace_size


def _norm(kind, name):
    code = NORMS.get(kind)
    if code is None:
        raise ValueError("%s must be one of %s, got %r" % (name, ", ".join(NORMS), kind))
    return code


def _dropped(p):
    """p as a number of 65536."""
    if not 0.0 <= p <= 1.0:
        raise ValueError("p must be between 0 and 1, got %r" % (p,))
    return int(p * 65536 + 0.5)


def _seed(seed, index):
    """The address of a seed in device memory and its value: one of the two."""
    if type(seed) is int and -2 ** 63 <= seed < 2 ** 63:
        return None, seed
    if isinstance(seed, _Tensor):
        if seed.dtype is not torch.int64 or not seed.is_cuda:
            raise TypeError("seed must be a number or a one-element int64 CUDA tensor")
        if seed.numel() != 1:
            raise ValueError("seed must have one element")
        if seed.get_device() != index:
            raise ValueError("seed must be on the device of the other tensors")
        return seed.data_ptr(), 0
    return None, _int64(seed, "seed")


def _int64(v, name):
    """v modulo 2^64 as a signed number."""
    if type(v) is int and -2 ** 63 <= v < 2 ** 63:
        return v
    if not isinstance(v, int):
        raise TypeError("%s must be an integer" % name)
    v &= 2 ** 64 - 1
    return v - 2 ** 64 if v >> 63 else v


def _gate(gate, dtype, index, M, N):
    """A gate's pointer, row stride and rows."""
    if gate is None:
        return None, N, 1
    if isinstance(gate, _Tensor) and gate.dim() == 2:
        rows = gate.shape[0]
        if rows == 0 or M % rows:
            raise ValueError("gate must have rows for equal numbers of the %d rows, got %s" % (M, tuple(gate.shape)))
        return (*_matrix(gate, "gate", dtype, index, (rows, N)), rows)
    return _vector(gate, "gate", dtype, index, N), N, 1


def _check(h, norm, weight, bias, gate, scale, post, post_weight, post_bias, p):
    if norm == binding.T2S_NORM_NONE and (weight is not None or bias is not None):
        raise ValueError("weight and bias need a norm")
    if post == binding.T2S_NORM_NONE and (post_weight is not None or post_bias is not None):
        raise ValueError("post_weight and post_bias need a post_norm")
    if h is None and (post != binding.T2S_NORM_NONE or gate is not None or p != 0 or scale != 1):
        raise ValueError("a post_norm, a gate, dropout and a scale need h")


def residual_norm(x, h=None, weight=None, bias=None, gate=None, scale=1.0, norm="rms", eps=1e-6, post_norm="none",
                  post_weight=None, post_bias=None, p=0.0, seed=0, sequence=0, r=None, y=None, stream=None):
    """(r, y): the residual stream after a block with output h, and the norm of it. With ``norm`` "none" y
    is None; without h only y is computed, the norm of x, and r is x itself. ``r`` and ``y`` are tensors to
    write to; r may be x."""
    dtype, device, index, xp, ldx, M, N = _first(x, "x")
    code, post = _norm(norm, "norm"), _norm(post_norm, "post_norm")
    dropped = _dropped(p)
    _check(h, code, weight, bias, gate, scale, post, post_weight, post_bias, p)
    hp, ldh = (None, N) if h is None else _matrix(h, "h", dtype, index, (M, N))
    gp, ldg, gates = _gate(gate, dtype, index, M, N)
    wp = None if weight is None else _vector(weight, "weight", dtype, index, N)
    bp = None if bias is None else _vector(bias, "bias", dtype, index, N)
    pw = None if post_weight is None else _vector(post_weight, "post_weight", dtype, index, N)
    pb = None if post_bias is None else _vector(post_bias, "post_bias", dtype, index, N)
    if _grad_enabled():
        for t in (x, h, weight, bias, gate, post_weight, post_bias):
            if t is not None and t.requires_grad:
                _refuse_history("residual_norm")
    if h is None:
        if code == binding.T2S_NORM_NONE:
            raise ValueError("without h there must be a norm")
        if r is not None:
            raise ValueError("without h, r is x")
        r, rp, ldr = x, None, N
    elif r is None:
        r = _new((M, N), (N, 1), dtype, device, stream)
        rp, ldr = r.data_ptr(), N
    else:
        rp, ldr = _matrix(r, "r", dtype, index, (M, N))
    if code == binding.T2S_NORM_NONE:
        if y is not None:
            raise ValueError("y needs a norm")
        yp, ldy = None, N
    elif y is None:
        y = _new((M, N), (N, 1), dtype, device, stream)
        yp, ldy = y.data_ptr(), N
    else:
        yp, ldy = _matrix(y, "y", dtype, index, (M, N))
    at, seed = _seed(seed, index)
    f = _FUNCTIONS.get(("t2s_residual_norm", dtype)) or _function("t2s_residual_norm", dtype)
    rc = f(M, N, code, post, xp, ldx, hp, ldh, wp, bp, pw, pb, gp, ldg, gates, scale, eps, dropped, at, seed,
           _int64(sequence, "sequence"), rp, ldr, yp, ldy, _raw_stream(index) if stream is None else stream)
    if rc != T2S_OK:
        raise T2SError(rc, "t2s_residual_norm" + _SUFFIX[dtype])
    return r, y


def residual_norm_backward(dy, dr, r, h=None, weight=None, bias=None, gate=None, scale=1.0, norm="rms", eps=1e-6,
                           post_norm="none", post_weight=None, post_bias=None, p=0.0, seed=0, sequence=0, dx=None,
                           dh=None, workspace=None, stream=None):
    """ResidualNormGradients from dy, the gradient of y (None with ``norm`` "none"), dr, that of r's other uses
    (None for none), r as the forward pass returned it, and the forward pass's other arguments. dx and dh
    are None (allocated here), tensors that receive them, or False (not computed); every parameter that
    is given gets its gradient. Those of vectors are contiguous; that of a matrix of gates has rows on
    16-byte boundaries, N rounded up to a multiple of 8 values apart."""
    code, post = _norm(norm, "norm"), _norm(post_norm, "post_norm")
    dtype, device, index, rp, ldr, M, N = _first(r, "r")
    if (dy is None) != (code == binding.T2S_NORM_NONE):
        raise ValueError("dy is needed with a norm, and only there")
    _check(h, code, weight, bias, gate, scale, post, post_weight, post_bias, p)
    dropped = _dropped(p)
    dyp, lddy = (None, N) if dy is None else _matrix(dy, "dy", dtype, index, (M, N))
    drp, lddr = (None, N) if dr is None else _matrix(dr, "dr", dtype, index, (M, N))
    hp, ldh = (None, N) if h is None else _matrix(h, "h", dtype, index, (M, N))
    gp, ldg, gates = _gate(gate, dtype, index, M, N)
    wp = None if weight is None else _vector(weight, "weight", dtype, index, N)
    if bias is not None:
        _vector(bias, "bias", dtype, index, N)
    pw = None if post_weight is None else _vector(post_weight, "post_weight", dtype, index, N)
    pb = None if post_bias is None else _vector(post_bias, "post_bias", dtype, index, N)
    dx, dxp, lddx = _output(dx, "dx", dtype, device, (M, N), stream)
    dh, dhp, lddh = (False, None, N) if h is None else _output(dh, "dh", dtype, device, (M, N), stream)
    grads, ptrs, ldgate, vectors = [None] * 5, [None] * 5, N, 0
    for j, t in enumerate((weight, bias, post_weight, post_bias)):
        if t is not None:
            grads[j] = t = _new((N,), (1,), dtype, device, stream)
            ptrs[j] = t.data_ptr()
            vectors += 1
    if gate is not None:
        if gate.dim() == 1:
            grads[4] = t = _new((N,), (1,), dtype, device, stream)
        else:
            ldgate = N + 7 & -8  # rows on 16-byte boundaries
            grads[4] = t = _new((gates, N), (ldgate, 1), dtype, device, stream)
        ptrs[4] = t.data_ptr()
        vectors += 1
    need = 0 if workspace is not None or not vectors or not M else (
        _workspace_size or _function_of_size())(M, N, gates, vectors)
    keep, ws, size = _workspace(workspace, need, device, stream)
    at, seed = _seed(seed, index)
    f = _FUNCTIONS.get(("t2s_residual_norm_backward", dtype)) or _function("t2s_residual_norm_backward", dtype)
    rc = f(M, N, code, post, dyp, lddy, drp, lddr, rp, ldr, hp, ldh, wp, pw, pb, gp, ldg, gates, scale, eps, dropped,
           at, seed, _int64(sequence, "sequence"), dxp, lddx, dhp, lddh, *ptrs, ldgate, ws, size,
           _raw_stream(index) if stream is None else stream)
    if rc != T2S_OK:
        raise T2SError(rc, "t2s_residual_norm_backward" + _SUFFIX[dtype])
    return ResidualNormGradients(None if dx is False else dx, None if dh is False else dh, grads[0], grads[1],
                                 grads[4], grads[2], grads[3])


def dropout(x, p, seed=0, sequence=0, residual=None, out=None, stream=None):
    """x with each value dropped with probability p and the others divided by 1 - p, plus ``residual``. ``out``
    may be x or the residual."""
    dtype, device, index, xp, ldx, M, N = _first(x, "x")
    dropped = _dropped(p)
    rp, ldr = (None, N) if residual is None else _matrix(residual, "residual", dtype, index, (M, N))
    if _grad_enabled() and (x.requires_grad or (residual is not None and residual.requires_grad)):
        _refuse_history("dropout")
    if out is None:
        out = _new((M, N), (N, 1), dtype, device, stream)
        yp, ldy = out.data_ptr(), N
    else:
        yp, ldy = _matrix(out, "out", dtype, index, (M, N))
    at, seed = _seed(seed, index)
    f = _FUNCTIONS.get(("t2s_dropout", dtype)) or _function("t2s_dropout", dtype)
    rc = f(M, N, xp, ldx, rp, ldr, dropped, at, seed, _int64(sequence, "sequence"), yp, ldy,
           _raw_stream(index) if stream is None else stream)
    if rc != T2S_OK:
        raise T2SError(rc, "t2s_dropout" + _SUFFIX[dtype])
    return out


def dropout_backward(dy, p, seed=0, sequence=0, dx=None, stream=None):
    """The gradient of ``dropout``'s x for its p, seed and sequence (the residual's is dy itself)."""
    return dropout(dy, p, seed, sequence, out=dx, stream=stream)
