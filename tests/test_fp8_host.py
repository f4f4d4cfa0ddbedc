"""The 8-bit operators' C ABI and checks without a GPU: bad arguments are refused before CUDA is touched."""
from __future__ import annotations

import pytest

torch = pytest.importorskip("torch")

from roofline_driven_tiling_gb300 import binding, fp8  # noqa: E402

F = 1 << 20  # never dereferenced: every call below fails validation or has no work


@pytest.fixture(scope="module")
def lib():
    import __graft_entry__
    __graft_entry__.build()
    return binding.lib()


def _call(lib, fn, a, kw):
    assert set(kw) <= set(a)
    return {getattr(lib, fn + t)(*dict(a, **kw).values()) for t in ("_bf16", "_f16", "_f32")}


def test_quantize_arguments(lib):
    a = dict(M=256, N=300, X=F, ldx=300, format=0, square=0, Q=F + (1 << 20), ldq=304, S=F + (1 << 21), s_row=1, s_block=256,
             Qt=F + (1 << 22), ldqt=256, St=F + (1 << 23), st_row=1, st_block=300, stream=None)
    for kw in (dict(M=-1), dict(N=-1), dict(M=binding.T2S_MAX_DIM + 1), dict(format=2), dict(format=-1), dict(square=2),
               dict(X=None), dict(X=F + 1), dict(ldx=299), dict(ldq=299), dict(ldqt=255), dict(S=None), dict(St=None),
               dict(S=F + 2), dict(Q=None, Qt=None), dict(Q=F), dict(Qt=F), dict(Qt=F + (1 << 20)), dict(St=F + (1 << 21)),
               dict(s_row=-1), dict(s_block=-256), dict(s_row=0), dict(s_block=255), dict(s_row=2), dict(s_row=3, s_block=1, M=4, ldqt=256, N=600, ldx=600, ldq=608, st_block=600),
               dict(st_block=299), dict(square=1, s_row=1, s_block=1)):
        assert _call(lib, "t2s_quantize_fp8", a, kw) == {binding.T2S_ERR_INVALID}, kw
    for kw in (dict(M=0), dict(N=0), dict(M=0, X=None, Q=None, Qt=None)):
        assert _call(lib, "t2s_quantize_fp8", a, kw) == {binding.T2S_OK}, kw


def test_gemm_arguments(lib):
    a = dict(M=64, N=200, K=300, A=F, lda=304, format_a=0, SA=F + (1 << 20), sa_row=1, sa_block=64, B=F + (1 << 21), ldb=304,
             format_b=1, SB=F + (1 << 22), sb_row=1, sb_block=200, group=1, C=F + (1 << 23), ldc=200, stream=None)
    for kw in (dict(M=-1), dict(N=-1), dict(K=-1), dict(K=binding.T2S_MAX_DIM + 1), dict(format_a=2), dict(format_b=-1),
               dict(group=0), dict(group=64), dict(A=None), dict(B=None), dict(C=None), dict(SA=None), dict(SB=None),
               dict(A=F + 8), dict(B=F + (1 << 21) + 4), dict(lda=300), dict(lda=312), dict(ldb=299), dict(ldb=310), dict(ldc=199),
               dict(C=F + (1 << 23) + 1), dict(C=F), dict(C=F + (1 << 21)), dict(SA=F + 1), dict(SB=F + 2), dict(sa_row=-1),
               dict(sb_block=-1), dict(sa_block=binding.T2S_MAX_DIM + 1)):
        assert _call(lib, "t2s_gemm_fp8", a, kw) == {binding.T2S_ERR_INVALID}, kw
    for kw in (dict(M=0), dict(N=0), dict(M=0, A=None, C=None)):
        assert _call(lib, "t2s_gemm_fp8", a, kw) == {binding.T2S_OK}, kw


def test_scales_are_no_other_argument(lib):
    Q, S, Qt, St = F + (1 << 20), F + (1 << 21), F + (1 << 22), F + (1 << 23)
    a = dict(M=256, N=300, X=F, ldx=300, format=0, square=0, Q=Q, ldq=304, S=S, s_row=1, s_block=256, Qt=Qt, ldqt=256, St=St,
             st_row=1, st_block=300, stream=None)
    for kw in (dict(S=F), dict(S=Q), dict(S=Qt), dict(St=F), dict(St=Q), dict(St=Qt), dict(Qt=None, S=F), dict(Q=None, St=Qt)):
        assert _call(lib, "t2s_quantize_fp8", a, kw) == {binding.T2S_ERR_INVALID}, kw
    a = dict(M=64, N=200, K=300, A=F, lda=304, format_a=0, SA=Q, sa_row=1, sa_block=64, B=S, ldb=304, format_b=1, SB=Qt,
             sb_row=1, sb_block=200, group=1, C=St, ldc=200, stream=None)
    for kw in (dict(C=Q), dict(C=Qt)):
        assert _call(lib, "t2s_gemm_fp8", a, kw) == {binding.T2S_ERR_INVALID}, kw


def test_python_checks():
    x = torch.zeros(4, 128)
    q = x.to(torch.float8_e4m3fn)
    for call in (lambda: fp8.quantize_fp8(x), lambda: fp8.quantize_fp8(q), lambda: fp8.quantize_fp8(None),
                 lambda: fp8.gemm_fp8(q, x, q.t(), x), lambda: fp8.gemm_fp8(x, x, q.t(), x)):
        with pytest.raises(TypeError):
            call()
