"""Sums of very many terms of one sign in the feed-forward operators (GPU tests).

A tensor core's accumulator truncates, always towards zero, so its error grows with the terms it
takes. The operators' bound: pieces of at most 16384 terms, at most 2^-23 of the sum of magnitudes lost
for every 16 terms of a piece, and the pieces added in FP32. With operands of one sign the sum of
magnitudes is the sum itself, and an output is off by at most that and its one rounding.
"""
from __future__ import annotations

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import roofline_driven_tiling_gb300 as t2s  # noqa: E402
from roofline_driven_tiling_gb300 import binding  # noqa: E402

F16 = torch.float16
PIECE = 16384
U = 2.0 ** -11
COLUMNS = 40  # of an output that are compared, spread over its tiles


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()
    torch.cuda.set_device(0)
    assert binding.device_status() == binding.T2S_OK
    yield
    torch.cuda.empty_cache()


def positive(gen, rows, cols, scale):
    out = torch.empty(rows, cols, dtype=F16, device="cuda")
    step = max(1, (1 << 28) // cols)
    for r in range(0, rows, step):
        part = out[r:r + step]
        part.copy_(torch.rand(part.shape, generator=gen, device="cuda") * scale)
    return out


def within(got, want, terms):
    lost = min(terms, PIECE) / 16 * 2.0 ** -23 + -(-terms // PIECE) * 2.0 ** -23
    worst = float(((got.double() - want).abs() / want).max())
    assert worst <= lost * (1 + U) + U, "%.3g of the sum, bar %.3g" % (worst, lost * (1 + U) + U)


def spread(n):
    return torch.linspace(0, n - 1, COLUMNS, device="cuda").long().unique()


def products(a, b, chunk=1 << 18):
    """a @ b in float64 over pieces of the sum."""
    want = torch.zeros(a.shape[0], b.shape[1], dtype=torch.float64, device="cuda")
    for k in range(0, a.shape[1], chunk):
        want += a[:, k:k + chunk].double() @ b[k:k + chunk].double()
    return want


@pytest.mark.parametrize("wt", [False, True])
def test_linear(wt):
    m, k, n = 1024, (1 << 21) + 24, 1000
    gen = torch.Generator(device="cuda").manual_seed(1)
    x = positive(gen, m, k, 2.0 ** -2)
    w = positive(gen, n, k, 2.0 ** -8).t() if wt else positive(gen, k, n, 2.0 ** -8)
    y = t2s.linear(x, w)
    assert binding.device_status() == binding.T2S_OK
    at = spread(n)
    within(y[:, at], products(x, w[:, at]), k)


@pytest.mark.parametrize("m", [3, 700])
def test_few_outputs(m):
    """Few tiles: the sum is split over a cluster where that leaves each CTA few enough terms."""
    k, n = (1 << 21) + 40, 72
    gen = torch.Generator(device="cuda").manual_seed(2)
    x, w, w2 = positive(gen, m, k, 2.0 ** -2), positive(gen, k, n, 2.0 ** -8), positive(gen, k, n, 2.0 ** -8)
    within(t2s.linear(x, w), products(x, w), k)
    g, u = torch.empty(m, n, dtype=F16, device="cuda"), torch.empty(m, n, dtype=F16, device="cuda")
    t2s.gated_linear(x, w, w2, act="relu", preact=(g, u))
    assert binding.device_status() == binding.T2S_OK
    within(g, products(x, w), k)
    within(u, products(x, w2), k)


def test_gated():
    m, k, n = 1024, 1 << 20, 1000
    gen = torch.Generator(device="cuda").manual_seed(3)
    x, wg, wu = (positive(gen, m, k, 2.0 ** -2), positive(gen, n, k, 2.0 ** -8).t(),
                 positive(gen, n, k, 2.0 ** -8).t())
    g, u = torch.empty(m, n, dtype=F16, device="cuda"), torch.empty(m, n, dtype=F16, device="cuda")
    t2s.gated_linear(x, wg, wu, act="relu", preact=(g, u))
    assert binding.device_status() == binding.T2S_OK
    at = spread(n)
    within(g[:, at], products(x, wg[:, at]), k)
    within(u[:, at], products(x, wu[:, at]), k)


def test_gradient_of_the_input():
    """dX = dG Wg^T + dU Wu^T is one sum of 2 N terms; pre-activations of 1 make dG = dU = dH."""
    m, k, n = 1000, 1040, (1 << 19) + 16
    gen = torch.Generator(device="cuda").manual_seed(4)
    dh, wg, wu = positive(gen, m, n, 2.0 ** -2), positive(gen, k, n, 2.0 ** -8), positive(gen, k, n, 2.0 ** -8)
    one = torch.ones(m, n, dtype=F16, device="cuda")
    dx, _, _ = t2s.gated_linear_backward(dh, positive(gen, m, k, 1.0), wg, wu, (one, one), act="relu", dw_gate=False,
                                         dw_up=False)
    assert binding.device_status() == binding.T2S_OK
    at = spread(k)
    within(dx[:, at], products(dh, wg[at].t()) + products(dh, wu[at].t()), 2 * n)


@pytest.mark.parametrize("k,n", [(1552, 1552), (264, 136)])
@pytest.mark.parametrize("wt", [False, True])
def test_gradients_of_weights(k, n, wt):
    """Over many rows: more tiles than pieces are cut for, and few enough that they are."""
    m = (1 << 20) + 40
    gen = torch.Generator(device="cuda").manual_seed(5)
    x, dy = positive(gen, m, k, 2.0 ** -2), positive(gen, m, n, 2.0 ** -8)
    w = torch.zeros(n, k, dtype=F16, device="cuda").t() if wt else torch.zeros(k, n, dtype=F16, device="cuda")
    _, dw, _ = t2s.linear_backward(dy, x, w, dx=False)
    assert binding.device_status() == binding.T2S_OK
    at = spread(n)
    within(dw[:, at], products(x.t(), dy[:, at]), m)
