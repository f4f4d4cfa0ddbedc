"""The feed-forward operators and torch's autograd (GPU tests): they record no history, so a forward call that
would lose a gradient is refused rather than cut out of the graph."""
from __future__ import annotations

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import roofline_driven_tiling_gb300 as t2s  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()
    torch.cuda.set_device(0)


def tensors(seed=0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return [torch.randn(*shape, generator=gen, device="cuda").bfloat16() for shape in ((9, 16), (16, 24), (24,), (9, 24))]


@pytest.mark.parametrize("which", range(4))
def test_linear_refuses_to_lose_a_gradient(which):
    args = tensors()
    want = t2s.linear(*args, act="silu")
    args[which].requires_grad_()
    with pytest.raises(ValueError, match="linear_backward"):
        t2s.linear(*args, act="silu")
    with torch.no_grad():
        assert torch.equal(t2s.linear(*args, act="silu"), want)
    with torch.inference_mode():
        assert torch.equal(t2s.linear(*args, act="silu"), want)


@pytest.mark.parametrize("which", range(3))
def test_gated_refuses_to_lose_a_gradient(which):
    x, w, _, _ = tensors()
    args = [x, w, w.clone()]
    want = t2s.gated_linear(*args)
    args[which].requires_grad_()
    with pytest.raises(ValueError, match="gated_linear_backward"):
        t2s.gated_linear(*args)
    with torch.no_grad():
        assert torch.equal(t2s.gated_linear(*args), want)


def test_gradients_take_parameters():
    """The backward functions are the history's place: leaves are what they are called with."""
    x, w, _, dy = tensors()
    want = t2s.linear_backward(dy, x, w)
    got = t2s.linear_backward(dy, x, w.clone().requires_grad_())
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]) and not got[0].requires_grad
