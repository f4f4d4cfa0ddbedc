"""The norms' and dropout's definitions without a GPU: formulas against differences, the mask against the
pinned generator, and refusals of bad arguments before CUDA is touched."""
from __future__ import annotations

import math

import pytest

torch = pytest.importorskip("torch")

import norm_reference as ref  # noqa: E402
from roofline_driven_tiling_gb300 import binding, norm  # noqa: E402


@pytest.fixture(scope="module")
def lib():
    import __graft_entry__
    __graft_entry__.build()
    return binding.lib()


@pytest.mark.parametrize("kind,post,gates", [("rms", "none", 0), ("layer", "rms", 1), ("rms", "layer", 3),
                                             ("none", "rms", 1), ("layer", "layer", 6)])
def test_formulas_are_the_differences(kind, post, gates):
    """Central differences of sum(r * u + y * v) with a step of 1e-6: truncation about 1e-12, rounding 1e-10."""
    gen = torch.Generator().manual_seed(3)

    def normal(*shape):
        return torch.randn(*shape, generator=gen, dtype=torch.float64)

    rows, cols = 6, 5
    x, h, u, v = (normal(rows, cols) for _ in range(4))
    tensors = {"weight": normal(cols), "bias": normal(cols)} if kind != "none" else {}
    if post != "none":
        tensors.update(post_weight=normal(cols), post_bias=normal(cols))
    if gates:
        tensors["gate"] = normal(cols) if gates == 1 else normal(gates, cols)
    keep = ref.factors(rows, cols, 0.3, 7, 2)

    def loss(x, h, **t):
        case = ref.Case(kind, post, 1e-3, 0.7, keep, **t)
        r = case.stream(x, h)
        return float((r * u).sum() + (0.0 if kind == "none" else (case.y(r) * v).sum()))

    case = ref.Case(kind, post, 1e-3, 0.7, keep, **tensors)
    got = case.gradients(None if kind == "none" else v, u, case.stream(x, h), h)
    for name, t in dict(tensors, x=x, h=h).items():
        want = torch.zeros_like(t)
        for i in range(t.numel()):
            side = []
            for step in (1e-6, -1e-6):
                moved = t.clone()
                moved.view(-1)[i] += step
                side.append(loss(**dict(dict(tensors, x=x, h=h), **{name: moved})))
            want.view(-1)[i] = (side[0] - side[1]) / 2e-6
        assert torch.allclose(got["d" + name].view(t.shape), want, rtol=1e-7, atol=1e-7), name


def test_mask():
    """The share of dropped values within five deviations, and no two sequences or seeds alike."""
    rows, cols, p = 64, 1001, 0.3
    masks = [ref.factors(rows, cols, p, seed, seq) == 0 for seed, seq in ((1, 0), (1, 1), (2, 0), (-1, 0), (1, 2 ** 63))]
    n = rows * cols
    for i, m in enumerate(masks):
        assert abs(int(m.sum()) - p * n) < 5 * math.sqrt(n * p * (1 - p))
        for other in masks[:i]:
            both = int((m & other).sum())
            assert abs(both - p * p * n) < 5 * math.sqrt(n * p * p)
    assert bool((ref.factors(8, 8, 0.0, 1, 1) == 1).all()) and bool((ref.factors(8, 8, 1.0, 1, 1) == 0).all())


def _call(lib, fn, a, kw):
    assert set(kw) <= set(a)
    return [getattr(lib, fn + t)(*dict(a, **kw).values()) for t in ("_bf16", "_f16")]


BAD, OK, SMALL = [binding.T2S_ERR_INVALID] * 2, [binding.T2S_OK] * 2, [binding.T2S_ERR_WORKSPACE] * 2
F = 1 << 20  # never dereferenced: every call below fails validation or has no work


def test_forward_arguments(lib):
    a = dict(M=4, N=8, norm=1, post=1, X=F, ldx=8, H=F + 4096, ldh=8, weight=F + 8192, bias=None, pw=F + 12288, pb=None,
             gate=F + 16384, ldgate=8, gates=2, scale=0.5, eps=1e-6, dropped=0, at=None, seed=1, sequence=0, R=F + 20480,
             ldr=8, Y=F + 24576, ldy=8, stream=None)
    for kw in (dict(M=-1), dict(N=-1), dict(N=binding.T2S_MAX_DIM + 1), dict(norm=3), dict(norm=-1), dict(post=3),
               dict(X=None), dict(X=F + 1), dict(ldx=7), dict(H=F + 4097), dict(ldh=7), dict(weight=F + 8193),
               dict(gate=F + 16385), dict(ldgate=7), dict(gates=0), dict(gates=3), dict(gates=-1), dict(scale=math.inf),
               dict(scale=math.nan), dict(eps=-1e-6), dict(eps=math.nan), dict(eps=math.inf), dict(dropped=-1),
               dict(dropped=65537), dict(at=F + 4), dict(R=None), dict(Y=None), dict(R=F + 4096), dict(Y=F), dict(Y=F + 4096),
               dict(Y=F + 20480), dict(Y=F + 16384), dict(Y=F + 8192), dict(R=F, ldr=9), dict(ldr=7), dict(ldy=7),
               dict(norm=0), dict(norm=0, weight=None), dict(post=0), dict(post=0, pw=None, pb=F),
               dict(H=None), dict(H=None, post=0, pw=None), dict(R=F, X=F, H=F)):
        assert _call(lib, "t2s_residual_norm", a, kw) == BAD, kw
    alone = dict(H=None, post=0, pw=None, gate=None, gates=1, scale=1.0, R=None)
    for kw in (dict(R=F + 20480), dict(scale=0.5), dict(dropped=1), dict(gate=F + 16384), dict(Y=None), dict(Y=F),
               dict(norm=0, weight=None, Y=None)):
        assert _call(lib, "t2s_residual_norm", a, dict(alone, **kw)) == BAD, kw
    assert _call(lib, "t2s_residual_norm", a, dict(M=0)) == OK == _call(lib, "t2s_residual_norm", a, dict(N=0))


def test_matrices_without_values_have_no_address(lib):
    a = dict(M=0, N=8, norm=1, post=1, X=None, ldx=8, H=None, ldh=8, weight=F + 8192, bias=None, pw=F + 12288, pb=None,
             gate=F + 16384, ldgate=8, gates=1, scale=0.5, eps=1e-6, dropped=7, at=None, seed=1, sequence=0, R=None,
             ldr=8, Y=None, ldy=8, stream=None)
    nothing = dict(M=4, N=0, weight=None, pw=None, gate=None)
    for kw in (dict(), dict(gates=5), dict(R=F), nothing, dict(M=0, N=0, norm=2)):
        assert _call(lib, "t2s_residual_norm", a, kw) == OK, kw


def test_backward_arguments(lib):
    a = dict(M=4, N=8, norm=1, post=1, dY=F, lddy=8, dR=F + 4096, lddr=8, R=F + 8192, ldr=8, H=F + 12288, ldh=8,
             weight=F + 16384, pw=F + 20480, pb=None, gate=F + 24576, ldgate=8, gates=2, scale=0.5, eps=1e-6, dropped=0,
             at=None, seed=1, sequence=0, dX=F + 28672, lddx=8, dH=F + 32768, lddh=8, dw=F + 36864, db=None,
             dpw=F + 40960, dpb=None, dgate=F + 45056, lddgate=8, ws=F, size=0, stream=None)
    fn = "t2s_residual_norm_backward"
    for kw in (dict(M=-1), dict(norm=3), dict(post=-1), dict(dY=None), dict(R=None), dict(dY=F + 1), dict(lddy=7),
               dict(ldr=7), dict(lddr=7), dict(gates=3), dict(gates=0), dict(dropped=65537), dict(eps=-1.0), dict(dX=F),
               dict(dX=F + 4096), dict(dX=F + 8192), dict(dH=F + 12288), dict(dH=F + 28672), dict(dw=F + 16384),
               dict(dpw=F + 36864), dict(dgate=F + 24576), dict(dw=F + 36865), dict(lddgate=7), dict(lddx=7),
               dict(norm=0), dict(norm=0, dY=None), dict(norm=0, dY=None, weight=None), dict(post=0), dict(post=0, pw=None),
               dict(H=None), dict(scale=math.nan), dict(at=F + 4)):
        assert _call(lib, fn, a, kw) == BAD, kw
    need = binding.t2s_residual_norm_backward_workspace_size(4, 8, 2, 3)
    assert need >= 2 * 3 * 8 * 4
    for kw in (dict(), dict(ws=None, size=need), dict(size=need // 256 * 256 - 256), dict(ws=F + 16, size=need)):
        assert _call(lib, fn, a, kw) == SMALL, kw
    assert _call(lib, fn, a, dict(N=0)) == OK


def test_workspace_sizes(lib):
    f = binding.t2s_residual_norm_backward_workspace_size
    assert f(0, 8, 1, 3) == 0 == f(8, 0, 1, 3) == f(8, 8, 1, 0) == f(-1, 8, 1, 1) == f(8, 8, 0, 1) == f(8, 8, 3, 1) == f(8, 8, 1, 6)
    for M, N, gates, vectors in ((1, 1, 1, 1), (1300, 1003, 4, 5), (1 << 20, 1 << 14, 1, 5), (4096, 64, 4096, 2)):
        assert f(M, N, gates, vectors) % 256 == 0 and 4 * N * vectors <= f(M, N, gates, vectors) <= 2000 * 4 * N * vectors + 256


def test_dropout_arguments(lib):
    a = dict(M=4, N=8, X=F, ldx=8, R=None, ldr=8, dropped=100, at=None, seed=1, sequence=0, Y=F + 4096, ldy=8, stream=None)
    for kw in (dict(M=-1), dict(N=-1), dict(X=None), dict(Y=None), dict(X=F + 1), dict(Y=F + 4097), dict(ldx=7), dict(ldy=7),
               dict(R=F + 8193), dict(R=F + 8192, ldr=7), dict(dropped=-1), dict(dropped=65537), dict(at=F + 2),
               dict(Y=F, ldy=9), dict(R=F + 4096, ldr=9), dict(X=F + 4096, ldx=9)):
        assert _call(lib, "t2s_dropout", a, kw) == BAD, kw
    assert _call(lib, "t2s_dropout", a, dict(M=0)) == OK == _call(lib, "t2s_dropout", a, dict(N=0, X=None, Y=None))


def test_python_checks():
    """What needs no device: numbers, names and combinations."""
    assert norm._dropped(0.0) == 0 and norm._dropped(1) == 65536 and norm._dropped(0.1) == 6554
    for p in (-0.1, 1.1, math.nan):
        with pytest.raises(ValueError):
            norm._dropped(p)
    assert norm._int64(-1, "seed") == -1 == norm._int64(2 ** 64 - 1, "seed") and norm._int64(2 ** 63, "s") == -2 ** 63
    with pytest.raises(TypeError):
        norm._int64(1.5, "seed")
    with pytest.raises(ValueError):
        norm._norm("batch", "norm")
    for t in (torch.zeros(1), torch.zeros(1, dtype=torch.int64)):
        with pytest.raises(TypeError):
            norm._seed(t, 0)
    with pytest.raises(TypeError):
        norm.dropout(torch.zeros(2, 2, dtype=torch.bfloat16), 0.1)
    with pytest.raises(TypeError):
        norm.residual_norm(torch.zeros(2, 2, dtype=torch.bfloat16))
