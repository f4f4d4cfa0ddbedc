"""Weights' gradients over many rows where every sum is exact (GPU tests).

Small integers: all products and partial sums are integers below 2^24, exact in FP32 in any order, so a
gradient is the float64 result rounded to the type, equal bit for bit. A piece of the sum that is left
out, read twice or added to another's tile changes it.
"""
from __future__ import annotations

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import roofline_driven_tiling_gb300 as t2s  # noqa: E402
from roofline_driven_tiling_gb300 import binding  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()
    torch.cuda.set_device(0)
    assert binding.device_status() == binding.T2S_OK


# Rows around the fewest that are cut into pieces, remainders of one block and of one row, and weights
# of one tile, of a few and of ragged ones.
ROWS = [1023, 1024, 1025, 4100, 16400, 40001]
WEIGHTS = [(64, 64), (257, 131), (520, 768), (40, 1000)]


@pytest.mark.parametrize("m", ROWS)
@pytest.mark.parametrize("k,n", WEIGHTS)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_weight_gradients(m, k, n, dtype):
    gen = torch.Generator(device="cuda").manual_seed(m + k)

    def ints(rows, cols, lo=-2, hi=3):
        return torch.randint(lo, hi, (rows, cols), generator=gen, device="cuda").to(dtype)

    x, dy, z, up = ints(m, k), ints(m, n), ints(m, n, -1, 2), ints(m, n, -1, 2)
    xt = x.double().t()
    for wt in (False, True):
        w = ints(n, k).t() if wt else ints(k, n)
        _, dw, db = t2s.linear_backward(dy, x, w, dx=False, db=None)
        assert torch.equal(dw, (xt @ dy.double()).to(dtype))
        assert torch.equal(db, dy.double().sum(0).to(dtype))
        dx, dw, _ = t2s.linear_backward(dy, x, w, z, act="relu")
        d = dy.double() * (z > 0)
        assert torch.equal(dw, (xt @ d).to(dtype))
        assert torch.equal(dx, (d @ w.double().t()).to(dtype))
        dg, du = d * up.double(), dy.double() * z.double().clamp(min=0)
        dx, dwg, dwu = t2s.gated_linear_backward(dy, x, w, w, (z, up), act="relu")
        assert torch.equal(dwg, (xt @ dg).to(dtype))
        assert torch.equal(dwu, (xt @ du).to(dtype))
        assert torch.equal(dx, ((dg + du) @ w.double().t()).to(dtype))
        alone = t2s.gated_linear_backward(dy, x, w, w, (z, up), act="relu", dx=False, dw_gate=False)[2]
        assert torch.equal(alone, dwu)
    assert binding.device_status() == binding.T2S_OK
