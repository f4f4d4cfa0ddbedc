"""The feed-forward operators' activations value by value (GPU tests).

The bars are relative to the value, so that the tails count: with h half the distance between 16-bit
numbers at the value, h for the one rounding and 2^-15 of the value for its evaluation in FP32 (a fit
to 2^-19, and exponentials of arguments up to 100 whose own rounding is 2^-24 of the argument).
"""
from __future__ import annotations

import math

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import roofline_driven_tiling_gb300 as t2s  # noqa: E402
from roofline_driven_tiling_gb300 import binding  # noqa: E402

BF16, F16 = torch.bfloat16, torch.float16
BITS = {BF16: 8, F16: 11}
LEAST = {BF16: -133, F16: -24}  # log2 of the smallest subnormal


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()
    torch.cuda.set_device(0)
    assert binding.device_status() == binding.T2S_OK


def gelu64(z):
    """gelu(z) and its slope in float64, each term by itself accurate in the tail."""
    p = 0.5 * torch.special.erfcx(-z / math.sqrt(2)) * torch.exp(-z * z / 2)
    density = torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    return z * p, p + z * density


def half_step(v, dtype):
    e = torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -140))) - (BITS[dtype] - 1)
    return torch.exp2(e.clamp(min=LEAST[dtype]) - 1)


def check(got, want, dtype, relative=2.0 ** -15):
    bar = half_step(want, dtype) * (1 + 2.0 ** -10) + relative * want.abs()
    over = (got.double() - want).abs() / bar
    worst = int(over.argmax())
    assert float(over[worst]) <= 1, "%g instead of %g" % (float(got[worst]), float(want[worst]))


def numbers(dtype, lo, hi):
    """Every number of the type in [lo, hi], a multiple of 8 of them."""
    every = torch.arange(-(1 << 15), 1 << 15, device="cuda").to(torch.int16).view(dtype)
    z = every[(every >= lo) & (every <= hi)]
    return z[:z.numel() // 8 * 8].contiguous()


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("m", [1, 600])
def test_gelu(dtype, m):
    for lo, hi in ((-12, -2), (-2, -2.0 ** -6), (2.0 ** -6, 12)):
        z = numbers(dtype, lo, hi)
        n = z.numel()
        x, w = torch.zeros(m, 8, dtype=dtype, device="cuda"), torch.zeros(8, n, dtype=dtype, device="cuda")
        x[:, 0], w[0] = 1, z
        value, slope = gelu64(z.double())
        y = t2s.linear(x, w, act="gelu")
        for row in (0, m - 1):
            check(y[row], value, dtype)
        # dU = dH act(G) and dG = dH U act'(G) where the only other factors are ones.
        one, zz = torch.ones(1, n, dtype=dtype, device="cuda"), z.view(1, n).clone()
        _, dg, du = t2s.gated_linear_backward(one, x[:1], w, w, (zz, one), act="gelu", dx=False)
        check(du[0], value, dtype)
        _, _, db = t2s.linear_backward(one, x[:1], w, zz, act="gelu", dx=False, dw=False, db=None)
        # Around its zero at -0.75 the slope is a difference of two larger terms.
        far = (z < -1.5) | (z > 0)
        check(db[far], slope[far], dtype, 2.0 ** -13)
        check(dg[0][far], slope[far], dtype, 2.0 ** -13)
    assert binding.device_status() == binding.T2S_OK


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("act,lo", [("silu", -60), ("gelu_tanh", -8)])
def test_logistic_activations(dtype, act, lo):
    """Down to where their logistic factor is 2^-87 and 2^-72; slopes but around their zeros."""
    for first, last in ((lo, -2), (-2, -2.0 ** -6), (2.0 ** -6, 12)):
        z = numbers(dtype, first, last)
        n, z64 = z.numel(), z.double()
        c, a = math.sqrt(2 / math.pi), 0.044715
        v, dv = (z64, 1.0) if act == "silu" else (2 * c * (z64 + a * z64 ** 3), 2 * c * (1 + 3 * a * z64 ** 2))
        s = torch.sigmoid(v)
        value, slope = z64 * s, s + z64 * s * torch.sigmoid(-v) * dv
        x, w = torch.zeros(1, 8, dtype=dtype, device="cuda"), torch.zeros(8, n, dtype=dtype, device="cuda")
        x[:, 0], w[0] = 1, z
        check(t2s.linear(x, w, act=act)[0], value, dtype)
        one, zz = torch.ones(1, n, dtype=dtype, device="cuda"), z.view(1, n).clone()
        _, dg, du = t2s.gated_linear_backward(one, x, w, w, (zz, one), act=act, dx=False)
        check(du[0], value, dtype)
        if first != -2:
            check(dg[0], slope, dtype, 2.0 ** -13)
    assert binding.device_status() == binding.T2S_OK


@pytest.mark.parametrize("act", ["relu", "silu", "gelu", "gelu_tanh"])
def test_pre_activations_beyond_the_type(act):
    """A gate of -70000 is kept as -inf in binary16: its activation and slope are 0, forward and backward."""
    m, k, n = 20, 64, 72
    gen = torch.Generator(device="cuda").manual_seed(1)
    x = torch.rand(m, k, generator=gen, device="cuda").to(F16) + 1
    wg = torch.randn(k, n, generator=gen, device="cuda").to(F16)
    wg[:, 5] = -2000
    wu = torch.randn(k, n, generator=gen, device="cuda").to(F16)
    g, u = torch.empty(m, n, dtype=F16, device="cuda"), torch.empty(m, n, dtype=F16, device="cuda")
    h = t2s.gated_linear(x, wg, wu, act=act, preact=(g, u))
    assert bool(torch.isneginf(g[:, 5]).all()) and bool((h[:, 5] == 0).all())
    dh = torch.randn(m, n, generator=gen, device="cuda").to(F16)
    dx, dwg, dwu = t2s.gated_linear_backward(dh, x, wg, wu, (g, u), act=act)
    assert bool((dwg[:, 5] == 0).all()) and bool((dwu[:, 5] == 0).all())
    # All gradients are those of a large finite gate.
    g2 = g.clone()
    g2[:, 5] = -60000
    for one, other in zip((dx, dwg, dwu), t2s.gated_linear_backward(dh, x, wg, wu, (g2, u), act=act)):
        assert bool(torch.isfinite(one).all()) and torch.equal(one, other)
    assert binding.device_status() == binding.T2S_OK
