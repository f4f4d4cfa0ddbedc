"""The feed-forward operators' C ABI without a GPU: bad arguments and workspaces are refused before
CUDA is touched, and the workspace sizes."""
from __future__ import annotations

import pytest

from roofline_driven_tiling_gb300 import binding


@pytest.fixture(scope="module")
def lib():
    import __graft_entry__
    __graft_entry__.build()
    return binding.lib()


def _linear(lib, **kw):
    fake = 1 << 20  # never dereferenced: every case below fails validation first, or has no work
    a = dict(M=4, N=8, K=16, X=fake, ldx=16, W=fake + 4096, ldw=8, order=0, bias=None, R=None, ldr=8, act=0,
             Y=fake + 8192, ldy=8, Z=None, ldz=8, ws=None, size=0, stream=None)
    assert set(kw) <= set(a)
    a.update(kw)
    return [f(*a.values()) for f in (lib.t2s_linear_bf16, lib.t2s_linear_f16)]


def test_linear_arguments(lib):
    fake, bad = 1 << 20, [binding.T2S_ERR_INVALID] * 2
    for kw in (dict(M=-1), dict(N=-1), dict(K=-1), dict(K=binding.T2S_MAX_DIM + 1), dict(X=None), dict(W=None),
               dict(Y=None), dict(X=fake + 1), dict(W=fake + 1), dict(Y=fake + 1), dict(bias=fake + 1), dict(Z=fake + 1),
               dict(ldx=15), dict(ldw=7), dict(ldy=7), dict(ldx=binding.T2S_MAX_DIM + 1), dict(order=1), dict(order=2),
               dict(order=-1), dict(act=5), dict(act=-1), dict(Y=fake), dict(Y=fake + 4096), dict(Z=fake),
               dict(Z=fake + 8192), dict(R=fake + 9000, ldr=7), dict(R=fake + 9001),
               dict(R=fake + 8192, ldr=9), dict(bias=fake + 8192), dict(Z=fake + 9000, ldz=7)):
        assert _linear(lib, **kw) == bad, kw
    ok = [binding.T2S_OK] * 2
    assert _linear(lib, M=0, X=None, Y=None) == ok
    assert _linear(lib, N=0, W=None, Y=None) == ok


def test_gated_and_gradient_arguments(lib):
    fake = 1 << 20

    def call(fn, a, kw):
        assert set(kw) <= set(a)
        return [getattr(lib, fn + t)(*dict(a, **kw).values()) for t in ("_bf16", "_f16")]

    bad, small, ok = [binding.T2S_ERR_INVALID] * 2, [binding.T2S_ERR_WORKSPACE] * 2, [binding.T2S_OK] * 2
    gated = dict(M=4, N=8, K=16, X=fake, ldx=16, Wg=fake + 4096, ldwg=8, Wu=fake + 8192, ldwu=8, order=0, act=2,
                 H=fake + 12288, ldh=8, G=None, ldg=8, U=None, ldu=8, ws=None, size=0, stream=None)
    for kw in (dict(M=-1), dict(X=None), dict(Wg=None), dict(Wu=None), dict(H=None), dict(order=3), dict(act=9),
               dict(ldwu=7), dict(H=fake), dict(G=fake + 12288), dict(G=fake + 16384, U=fake + 16384),
               dict(U=fake + 1), dict(order=1)):
        assert call("t2s_gated", gated, kw) == bad, kw
    assert call("t2s_gated", gated, dict(M=0, X=None, H=None)) == ok
    back = dict(M=4, N=8, K=16, dY=fake, lddy=8, X=fake + 4096, ldx=16, W=fake + 8192, ldw=8, order=0, Z=fake + 12288,
                ldz=8, act=2, dX=fake + 16384, lddx=16, dW=fake + 20480, lddw=8, db=fake + 24576, ws=fake, size=0,
                stream=None)
    for kw in (dict(M=-1), dict(dY=None), dict(X=None), dict(W=None), dict(Z=None), dict(act=7), dict(lddy=7),
               dict(lddx=15), dict(lddw=7), dict(dX=fake), dict(dW=fake + 8192), dict(db=fake + 20480),
               dict(db=fake + 1), dict(order=1)):
        assert call("t2s_linear_backward", back, kw) == bad, kw
    need = binding.t2s_linear_backward_workspace_size(4, 8, 16, 1)
    for kw in (dict(), dict(ws=None, size=need), dict(size=need - 1), dict(ws=fake + 16, size=need)):
        assert call("t2s_linear_backward", back, kw) == small, kw
    both = dict(M=4, N=8, K=16, dH=fake, lddh=8, X=fake + 4096, ldx=16, Wg=fake + 8192, ldwg=8, Wu=fake + 12288, ldwu=8,
                order=0, G=fake + 16384, ldg=8, U=fake + 20480, ldu=8, act=2, dX=fake + 24576, lddx=16,
                dWg=fake + 28672, lddwg=8, dWu=fake + 32768, lddwu=8, ws=fake, size=0, stream=None)
    for kw in (dict(M=-1), dict(dH=None), dict(X=None), dict(Wg=None), dict(Wu=None), dict(G=None), dict(U=None),
               dict(act=7), dict(dX=fake), dict(dWg=fake + 32768), dict(dWu=fake + 8192), dict(ldu=7), dict(order=1)):
        assert call("t2s_gated_backward", both, kw) == bad, kw
    need = binding.t2s_gated_backward_workspace_size(4, 8, 16, 1)
    for kw in (dict(), dict(ws=None, size=need), dict(size=need - 1), dict(ws=fake + 16, size=need)):
        assert call("t2s_gated_backward", both, kw) == small, kw


def test_feed_forward_workspace_sizes(lib):
    f = binding
    # Aligned operands are read in place; the gradients keep dZ (dG, dU) there.
    assert f.t2s_linear_workspace_size(100, 200, 300, 1) == 0 == f.t2s_gated_workspace_size(100, 200, 300, 1)
    assert f.t2s_linear_workspace_size(4, 5, 7, 0) >= 2 * (4 * 8 + 5 * 8)
    assert f.t2s_gated_workspace_size(4, 5, 7, 0) >= 2 * (4 * 8 + 2 * 7 * 8)
    assert f.t2s_linear_backward_workspace_size(64, 72, 80, 1) >= 2 * 64 * 72
    assert f.t2s_gated_backward_workspace_size(64, 72, 80, 1) >= 2 * 2 * 64 * 72
    # Small weights over many rows: pieces of their gradients' sums; partial sums of db.
    assert f.t2s_linear_backward_workspace_size(8192, 256, 512, 1) >= 2 * 8192 * 256 + 2 * 4 * 256 * 512
    assert f.t2s_gated_backward_workspace_size(8192, 256, 512, 1) >= 2 * 2 * 8192 * 256 + 2 * 2 * 4 * 256 * 512
    assert f.t2s_linear_backward_workspace_size(1 << 16, 64, 1, 1) > 2 * 64 * (1 << 16)
    for g in (f.t2s_linear_workspace_size, f.t2s_linear_backward_workspace_size, f.t2s_gated_workspace_size,
              f.t2s_gated_backward_workspace_size):
        assert g(-1, 2, 3, 0) == 0 and g(2, f.T2S_MAX_DIM + 1, 3, 0) == 0
        assert g(33, 35, 37, 0) % 256 == 0 and g(33, 35, 37, 0) >= g(33, 35, 37, 1)
        # Sizes of large problems do not wrap.
        assert g(1 << 17, 1 << 17, 1 << 17, 0) >= 2 << 34
