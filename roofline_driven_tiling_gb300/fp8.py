"""Products of 8-bit floating-point CUDA tensors with a scale for each block of 128.

    quantize_fp8   x in 8 bits along its rows, its columns (transposed) or both, and the scales
    gemm_fp8       C = sum over blocks b of 128 of K of a[:, b] b[b, :] times both operands' scales

An operand keeps its K values side by side: ``a`` is M x K with contiguous rows, ``b`` is K x N and
the transpose of a tensor with contiguous rows, each row on a 16-byte boundary (the results of
``quantize_fp8`` are laid out so). Scales are float32: M x ceil(K / 128) for ``a``, ceil(K / 128) x N
or (one for 128 x 128) ceil(K / 128) x ceil(N / 128) for ``b``. For a layer y = x w of an inputs x
outputs weight and its gradients, with weights scaled in 128 x 128:

    wt, wts = quantize_fp8(w, along="columns", square=True)     # kept: w in 8 bits, once each way
    wn, wns = quantize_fp8(w, along="rows", square=True)
    xq, xs = quantize_fp8(x)
    y = gemm_fp8(xq, xs, wt.t(), wts.t())
    dq, ds, dt, dts = quantize_fp8(dy, along="both")
    dx = gemm_fp8(dq, ds, wn.t(), wns.t())
    xt, xts = quantize_fp8(x, along="columns")
    dw = gemm_fp8(xt, xts, dt.t(), dts.t(), dtype=torch.float32)

Sums are FP32, outputs are rounded once. Scales lie below 2^89 in magnitude (those of ``quantize_fp8`` do for
values up to 2^96, with e5m2 2^103), and the products of the two that meet are finite.

The work runs on ``stream`` (the integer value of a cudaStream_t; default: torch's current stream). No
autograd history is recorded: tensors that require grad (8-bit ones do where they were cast from such a
tensor, or are parameters) are refused unless gradients are off (``torch.no_grad()``).
"""
from __future__ import annotations

import ctypes

import torch

from . import binding
from .binding import T2S_OK, T2SError
from .feed_forward import _current_device, _grad_enabled, _new, _raw_stream, _row_stride, _Tensor

_FORMATS = {torch.float8_e4m3fn: binding.T2S_E4M3, torch.float8_e5m2: binding.T2S_E5M2}
_QUANTIZE = {torch.bfloat16: "t2s_quantize_fp8_bf16", torch.float16: "t2s_quantize_fp8_f16",
             torch.float32: "t2s_quantize_fp8_f32"}
_GEMM = {torch.bfloat16: "t2s_gemm_fp8_bf16", torch.float16: "t2s_gemm_fp8_f16", torch.float32: "t2s_gemm_fp8_f32"}
_FUNCTIONS = {}


def _function(names, dtype):
    """The C entry point for a type; its arguments are all integers, converted as pointers (the quickest)."""
    f = _FUNCTIONS.get(names[dtype])
    if f is None:
        f = binding.lib()[names[dtype]]
        f.argtypes = [ctypes.c_void_p] * len(binding.SIGNATURES[names[dtype]][0])
        f.restype = ctypes.c_int
        _FUNCTIONS[names[dtype]] = f
    return f


def _on_device(t, name, index):
    if t.get_device() != index:
        raise ValueError("%s must be on the device of the other tensors" % name)


def _new_quantized(rows, cols, group, dtype, device, stream):
    """8-bit rows on 16-byte boundaries, and scales whose rows are neighbours, each block's on one too."""
    ld, blocks, groups = cols + 15 & -16, (cols + 127) // 128, (rows + group - 1) // group
    q = _new((rows, cols), (ld, 1), dtype, device, stream)
    return q, _new((groups, blocks), (1, groups + 3 & -4), torch.float32, device, stream)


def _given(out, name, shape, dtype, group, index):
    """A caller's pair of 8-bit values and scales, checked."""
    q, s = out
    rows, cols = shape
    for t, what, d in ((q, name, dtype), (s, "scales of " + name, torch.float32)):
        if not isinstance(t, _Tensor) or t.dtype is not d:
            raise TypeError("%s must be a %s CUDA tensor" % (what, d))
        _on_device(t, what, index)
    if tuple(q.shape) != (rows, cols):
        raise ValueError("%s must be %d x %d" % (name, rows, cols))
    want = ((rows + group - 1) // group, (cols + 127) // 128)
    if tuple(s.shape) != want:
        raise ValueError("scales of %s must be %d x %d" % (name, *want))
    return q, s


def quantize_fp8(x, dtype=torch.float8_e4m3fn, along="rows", square=False, out=None, stream=None):
    """x (2-D, bfloat16, float16 or float32) in 8 bits with the scales of its blocks.

    ``along`` "rows": (q, scale), q like x, scale rows x ceil(columns / 128). "columns": (q, scale) of
    x.t(), q columns x rows. "both": (q, scale, qt, scale_t) from one read. ``square``: a scale for
    128 x 128 values instead of 128 of a row. A scale is the least power of two, at least 2^-126,
    with which the block's largest magnitude does not pass the type's largest value; q * scale
    stands for x. ``out``: the tuple to write to, in that order."""
    if not isinstance(x, _Tensor) or x.dtype not in _QUANTIZE or x.get_device() < 0:
        raise TypeError("x must be a bfloat16, float16 or float32 CUDA tensor")
    form = _FORMATS.get(dtype)
    if form is None:
        raise ValueError("dtype must be torch.float8_e4m3fn or torch.float8_e5m2, got %r" % (dtype,))
    if along not in ("rows", "columns", "both"):
        raise ValueError('along must be "rows", "columns" or "both", got %r' % (along,))
    index = x.get_device()
    if index != _current_device():
        raise ValueError("x must be on the current CUDA device")
    if x.dim() != 2:
        raise ValueError("x must be 2-D")
    if x.requires_grad and _grad_enabled():
        raise ValueError("quantize_fp8 records no autograd history, and x requires grad: call it under torch.no_grad()")
    rows, cols = x.shape
    ldx = _row_stride(x, "x", rows, cols)
    group, device, pairs, got = 128 if square else 1, x.device, [None] * 10, []
    if out is not None and len(out) != (4 if along == "both" else 2):
        raise ValueError("out must hold %d tensors" % (4 if along == "both" else 2))
    for i, (way, shape) in enumerate((("columns", (rows, cols)), ("rows", (cols, rows)))):
        if along == way:  # only the other one
            continue
        name = "qt" if i else "q"
        q, s = (_new_quantized(*shape, group, dtype, device, stream) if out is None else
                _given(out[len(got):len(got) + 2], name, shape, dtype, group, index))
        got += [q, s]
        pairs[5 * i:5 * i + 5] = [q.data_ptr(), _row_stride(q, name, *shape), s.data_ptr(), *s.stride()]
    f = _FUNCTIONS.get(_QUANTIZE[x.dtype]) or _function(_QUANTIZE, x.dtype)
    rc = f(rows, cols, x.data_ptr(), ldx, form, 1 if square else 0, *pairs,
           _raw_stream(index) if stream is None else stream)
    if rc != T2S_OK:
        raise T2SError(rc, _QUANTIZE[x.dtype])
    return tuple(got)


def _check_scale(t, name, index):
    if not isinstance(t, _Tensor) or t.dtype is not torch.float32 or t.get_device() < 0:
        raise TypeError("%s must be a float32 CUDA tensor" % name)
    _on_device(t, name, index)


def gemm_fp8(a, a_scale, b, b_scale, dtype=torch.bfloat16, out=None, stream=None):
    """The product of 8-bit a (M x K) and b (K x N) with their scales, in ``dtype`` (bfloat16,
    float16 or float32); each operand is float8_e4m3fn or float8_e5m2."""
    if not isinstance(a, _Tensor) or a.dtype not in _FORMATS or a.get_device() < 0:
        raise TypeError("a must be a float8_e4m3fn or float8_e5m2 CUDA tensor")
    index = a.get_device()
    if index != _current_device():
        raise ValueError("a must be on the current CUDA device")
    if not isinstance(b, _Tensor) or b.dtype not in _FORMATS or b.get_device() < 0:
        raise TypeError("b must be a float8_e4m3fn or float8_e5m2 CUDA tensor")
    if dtype not in _GEMM:
        raise ValueError("dtype must be torch.bfloat16, torch.float16 or torch.float32, got %r" % (dtype,))
    if a.dim() != 2 or b.dim() != 2 or b.shape[0] != a.shape[1]:
        raise ValueError("shape mismatch: a %s, b %s" % (tuple(a.shape), tuple(b.shape)))
    (M, K), N = a.shape, b.shape[1]
    _on_device(b, "b", index)
    lda, (step, ldb) = _row_stride(a, "a", M, K), b.stride()
    if N <= 1:
        ldb = K + 15 & -16
    if (step != 1 and K > 1) or ldb < K:
        raise ValueError("b must be the transpose of a tensor with contiguous rows that do not overlap")
    if M <= 1:
        lda = K + 15 & -16
    ap, bp = a.data_ptr(), b.data_ptr()
    if (ap | bp | lda | ldb) & 15 and M and N and K:
        raise ValueError("rows of a and of b.t() must start on 16-byte boundaries")
    blocks = (K + 127) // 128
    _check_scale(a_scale, "a_scale", index)
    if a_scale.shape != (M, blocks):
        raise ValueError("a_scale must be %d x %d, got %s" % (M, blocks, tuple(a_scale.shape)))
    _check_scale(b_scale, "b_scale", index)
    group = 1 if b_scale.shape == (blocks, N) else 128
    if group == 128 and b_scale.shape != (blocks, (N + 127) // 128):
        raise ValueError("b_scale must be %d x %d or %d x %d, got %s" % (
            blocks, N, blocks, (N + 127) // 128, tuple(b_scale.shape)))
    if _grad_enabled() and (a.requires_grad or b.requires_grad or a_scale.requires_grad or b_scale.requires_grad):
        raise ValueError("gemm_fp8 records no autograd history, and an input requires grad: call it under torch.no_grad()")
    if out is None:
        out, ldc = _new((M, N), (N, 1), dtype, a.device, stream), N
    else:
        if not isinstance(out, _Tensor) or out.dtype is not dtype:
            raise TypeError("out must be a %s CUDA tensor" % dtype)
        _on_device(out, "out", index)
        if tuple(out.shape) != (M, N):
            raise ValueError("out must be %d x %d" % (M, N))
        ldc = _row_stride(out, "out", M, N)
    sa, (sb_block, sb_row) = a_scale.stride(), b_scale.stride()
    f = _FUNCTIONS.get(_GEMM[dtype]) or _function(_GEMM, dtype)
    rc = f(M, N, K, ap, lda, _FORMATS[a.dtype], a_scale.data_ptr(), sa[0], sa[1], bp, ldb, _FORMATS[b.dtype],
           b_scale.data_ptr(), sb_row, sb_block, group, out.data_ptr(), ldc,
           _raw_stream(index) if stream is None else stream)
    if rc != T2S_OK:
        raise T2SError(rc, _GEMM[dtype])
    return out
