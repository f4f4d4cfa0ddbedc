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


@pytest.mark.parametrize("k", [16383, 16384, 16385, 32768, 32776, 49160])
@pytest.mark.parametrize("m,n", [(1, 72), (24, 264), (300, 136), (520, 1100)])
def test_sums_around_an_accumulators_length(m, n, k):
    """16384 values go to one accumulator; a value more, and several accumulators' worth."""
    gen = torch.Generator(device="cuda").manual_seed(k)

    def ints(rows, cols):
        return torch.randint(-2, 3, (rows, cols), generator=gen, device="cuda").half()

    x, bias, r = ints(m, k), ints(1, n).reshape(n), ints(m, n)
    for wt in (False, True):
        w, w2 = [ints(n, k).t() if wt else ints(k, n) for _ in range(2)]
        z, z2 = x.double() @ w.double(), x.double() @ w2.double()
        kept, g, u = [torch.empty(m, n, dtype=torch.float16, device="cuda") for _ in range(3)]
        y = t2s.linear(x, w, bias, r, act="relu", preact=kept)
        assert torch.equal(kept, (z + bias.double()).half())
        assert torch.equal(y, ((z + bias.double()).clamp(min=0) + r.double()).half())
        h = t2s.gated_linear(x, w, w2, act="relu", preact=(g, u))
        assert torch.equal(g, z.half()) and torch.equal(u, z2.half())
        assert torch.equal(h, (z.clamp(min=0) * z2).half())
        # The joined gradient's two halves are one sum: dX = dH W^T + dH W2^T where G = U = 1.
        one = torch.ones(m, k // 2, dtype=torch.float16, device="cuda")
        a, b = [v[:k // 2].t() for v in (w, w2)]
        dx = t2s.gated_linear_backward(x[:, :k // 2], r, a, b, (one, one), act="relu", dw_gate=False, dw_up=False)[0]
        assert torch.equal(dx, (x[:, :k // 2].double() @ (w + w2)[:k // 2].double()).half())
    assert binding.device_status() == binding.T2S_OK


@pytest.mark.parametrize("m", [33000, 70001])
def test_pieces_longer_than_an_accumulator(m):
    """36 tiles of a weight leave room for two pieces, each longer than an accumulator takes from 32769 rows on."""
    k = n = 1536
    gen = torch.Generator(device="cuda").manual_seed(m)
    x, dy = [torch.randint(-2, 3, (m, k), generator=gen, device="cuda").half() for _ in range(2)]
    w = torch.zeros(k, n, dtype=torch.float16, device="cuda")
    want = (x.double().t() @ dy.double()).half()
    assert torch.equal(t2s.linear_backward(dy, x, w, dx=False)[1], want)
    assert torch.equal(t2s.linear_backward(dy, x, w.t())[1], want)
    assert binding.device_status() == binding.T2S_OK
