"""The feed-forward block on the package's operators (GPU tests): it learns, its gradients are the
block's, and single rows from a graph are the rows of a batch."""
from __future__ import annotations

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()
    torch.cuda.set_device(0)


def test_block_learns():
    from roofline_driven_tiling_gb300.block import FeedForwardBlock, train
    block, teacher = FeedForwardBlock(128, 320), FeedForwardBlock(128, 320, seed=1)
    x = torch.randn(600, 128, generator=torch.Generator(device="cuda").manual_seed(2), device="cuda").bfloat16()
    losses = train(block, x, teacher.forward(x), 20, 0.2)
    # Two independent blocks differ by about twice the branch's variance; descent at this rate
    # halves that several times within 20 steps.
    assert losses[-1] < 0.5 * losses[0], losses
    assert all(b < 1.05 * a for a, b in zip(losses, losses[1:])), losses


def test_block_gradients():
    """Against torch's own differentiation of the block in float64, on the same 16-bit weights. Relative
    2-norm: four roundings of intermediate values (h or G and U, dH, dG and dU, the result), each at most
    2^-8, and their spread through the products."""
    from roofline_driven_tiling_gb300.block import FeedForwardBlock
    block = FeedForwardBlock(96, 200, seed=3)
    gen = torch.Generator(device="cuda").manual_seed(4)
    x = torch.randn(77, 96, generator=gen, device="cuda").bfloat16()
    dy = torch.randn(77, 96, generator=gen, device="cuda").bfloat16()
    block.forward(x, keep=True)
    got = [block.backward(dy)[0], *block.backward(dy)[1]]
    leaves = [x.double().requires_grad_(), *[w.double().requires_grad_() for w in block.weights]]
    a, g, u, d = leaves
    y = a + (torch.nn.functional.silu(a @ g) * (a @ u)) @ d
    want = torch.autograd.grad(y, leaves, dy.double())
    for one, other in zip(got, want):
        assert float((one.double() - other).norm() / other.norm()) < 4 * 2.0 ** -8


def test_single_rows_from_a_graph():
    """One row takes another tiling than a batch: the sums' order differs, by FP32 rounding of sums, and a
    value near a rounding boundary may round the other way (twice: h and y)."""
    from roofline_driven_tiling_gb300.block import FeedForwardBlock, single_row
    block = FeedForwardBlock(256, 768, seed=5)
    x = torch.randn(300, 256, generator=torch.Generator(device="cuda").manual_seed(6), device="cuda").bfloat16()
    y = block.forward(x)
    graph, one, out = single_row(block, 256, torch.bfloat16)
    for i in (0, 1, 150, 299):
        one.copy_(x[i:i + 1])
        graph.replay()
        torch.cuda.synchronize()
        assert float((out.double() - y[i].double()).norm() / y[i].double().norm()) < 2 * 2.0 ** -8
