"""The feed-forward operators' activations value by value (GPU tests)."""
from __future__ import annotations

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import roofline_driven_tiling_gb300 as t2s  # noqa: E402
from roofline_driven_tiling_gb300 import binding  # noqa: E402

BF16, F16 = torch.bfloat16, torch.float16


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()
    torch.cuda.set_device(0)
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
