"""Norms and their gradients where rows are few or narrow for a block: groups of threads without a row, and rows of less
than a word, whose neighbours' words reach past the matrix (GPU tests).

A row's r, y, dx and dh, and dgate of a gate of its own, come from that row alone, so that they have the same bits in a
batch of any number of rows with the same places. Bars against float64 are those of test_norm_gpu."""
from __future__ import annotations

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import roofline_driven_tiling_gb300 as t2s  # noqa: E402
from roofline_driven_tiling_gb300 import binding  # noqa: E402
from test_norm_gpu import build, check_backward, check_forward, Maker  # noqa: E402

BF16, F16 = torch.bfloat16, torch.float16


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()
    torch.cuda.set_device(0)
    assert binding.device_status() == binding.T2S_OK


def tensors(m, n, dtype, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    new = lambda *s, mean=0.0: (mean + torch.randn(*s, generator=gen, device="cuda")).to(dtype)  # noqa: E731
    t = {name: new(m, n) for name in ("x", "h", "dy", "dr")}
    t["gate"] = new(m, n, mean=0.5)
    opt = dict(weight=new(n, mean=1.0), bias=new(n), norm="layer", post_norm="rms", post_weight=new(n, mean=1.0),
               post_bias=new(n), scale=0.5, eps=1e-5, p=0.2, seed=seed, sequence=3)
    return t, opt


def run(t, opt, rows, stream=None):
    """r, y and the gradients of the first rows, each with a gate of its own."""
    gate = t["gate"][:rows]
    r, y = t2s.residual_norm(t["x"][:rows], t["h"][:rows], gate=gate, stream=stream, **opt)
    g = t2s.residual_norm_backward(t["dy"][:rows], t["dr"][:rows], r, t["h"][:rows], gate=gate, stream=stream, **opt)
    return (r, y, g.dx, g.dh, g.dgate), (g.dweight, g.dbias, g.dpost_weight, g.dpost_bias)


@pytest.mark.parametrize("n", [8, 64, 96, 256, 257, 520, 1003, 2048, 4097])
def test_groups_without_a_row(n):
    """Fewer rows than a block has groups of threads, call after call on two streams, so that a block's memory goes to the
    next one at once: the bits of the same rows among many."""
    many = 3200  # rows for every group of every block
    t, opt = tensors(many, n, BF16, n)
    whole, _ = run(t, opt, many)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for rows in (1, 2, 3, 5, 9, 15):
        got = [run(t, opt, rows, s.cuda_stream) for _ in range(6) for s in streams]
        torch.cuda.synchronize()
        for own, sums in got:
            for a, b in zip(own, whole):
                assert bool((a == b[:rows]).all())
            for a, b in zip(sums, got[0][1]):
                assert bool((a == b).all())
        # One row: the sums over rows are its terms.
        if rows == 1:
            assert bool((got[0][1][1] == t["dy"][0]).all())
    assert binding.device_status() == binding.T2S_OK


@pytest.mark.parametrize("n", [1, 2, 3, 5, 6, 7, 9])
def test_many_narrow_rows(n):
    """More rows than all groups of a launch take at once, each of less than a word and up to seven of them in one."""
    for i, (dtype, pad, shift) in enumerate([(BF16, 0, 0), (F16, 0, 3), (BF16, 1, 5), (F16, 8, 1)]):
        m = 11000 + i
        mk = Maker(i, dtype, pad, shift)
        opt, t = build(mk, 6 * n + i, m, n)
        r, y = t2s.residual_norm(t["x"], t["h"], r=mk.empty(m, n), y=mk.empty(m, n), **opt)
        check_forward(opt, t["x"], t["h"], r, y, dtype, str(opt.keys()))
        dy, dr = mk.normal(m, n), mk.normal(m, n)
        g = t2s.residual_norm_backward(dy, dr, r, t["h"], dx=mk.empty(m, n), dh=mk.empty(m, n), **opt)
        check_backward(opt, dy, dr, r, t["h"], g, dtype, str(opt.keys()))
        mk.check_canaries()
    assert binding.device_status() == binding.T2S_OK


@pytest.mark.parametrize("n,pad,shift", [(4097, 0, 0), (4104, 1, 3), (5001, 0, 0), (6000, 3, 1), (8191, 0, 0), (8192, 0, 1), (8192, 0, 0)])
def test_sums_of_long_rows(n, pad, shift):
    """Rows of 4097 to 8192 values with all inputs and all sums are read once, as with fewer: dr of zeros gives the bits of no
    dr at all, which one reading and several passes over memory would not."""
    m = 333
    t, opt = tensors(m, n, BF16, n + shift)
    mk = Maker(1, BF16, pad, shift)

    def moved(v):
        view = mk.empty(m, n)
        view.copy_(v)
        return view

    h, dy, zero = moved(t["h"]), moved(t["dy"]), moved(torch.zeros(m, n))
    for gate in (t["gate"][0].clone(), t["gate"][:3].clone()):
        kw = dict(opt, gate=gate)
        r, _ = t2s.residual_norm(t["x"], h, **kw)
        far_r = moved(r)
        want = t2s.residual_norm_backward(dy, None, far_r, h, **kw)
        got = t2s.residual_norm_backward(dy, zero, far_r, h, **kw)
        check_backward(kw, dy, zero, far_r, h, got, BF16, str(n))
        for name, a, b in zip(got._fields, got, want):
            assert bool((a == b).all()), name
    assert binding.device_status() == binding.T2S_OK


@pytest.mark.parametrize("n", [8, 20, 1003])
def test_places_of_gate_gradients(n):
    """A vector's gradient is contiguous, a matrix's rows start on 16-byte boundaries."""
    t, opt = tensors(6, n, BF16, n)
    for gate, strides in ((t["gate"][0].clone(), (1,)), (t["gate"][:3], ((n + 7) // 8 * 8, 1))):
        g = t2s.residual_norm_backward(t["dy"], None, t["x"], t["h"], gate=gate, **opt)
        assert g.dgate.shape == gate.shape and g.dgate.stride() == strides and g.dgate.data_ptr() % 16 == 0
