"""Norms with residual and dropout, quantisation and 8-bit products as a block uses them, forward and backward:
each stage against its formula in float64 from the tensors that it really got (GPU tests). The bars are those
of the stages' own tests."""
from __future__ import annotations

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import norm_reference as ref  # noqa: E402
import roofline_driven_tiling_gb300 as t2s  # noqa: E402
from roofline_driven_tiling_gb300 import binding  # noqa: E402
from test_fp8_gpu import check_product, operand, quantized  # noqa: E402
from test_norm_gpu import check_backward, check_forward, reference, U, within  # noqa: E402

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
E4M3, E5M2 = torch.float8_e4m3fn, torch.float8_e5m2


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()
    torch.cuda.set_device(0)
    assert binding.device_status() == binding.T2S_OK


class Block:
    """r, y = residual_norm(x, h); z = y w in 8 bits; r2, y2 = residual_norm(r, z); out = dropout(y2); and all gradients.
    Weights and activations as one seed gives them; masks by the tensor `seed`."""

    def __init__(self, m, c, dtype, gates, seed):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        new = lambda *s, mean=0.0: (mean + torch.randn(*s, generator=gen, device="cuda")).to(dtype)  # noqa: E731
        self.m, self.c, self.dtype = m, c, dtype
        self.x, self.h, self.dout = new(m, c), new(m, c), new(m, c)
        self.w = torch.randn(c, c, generator=gen, device="cuda") * c ** -0.5
        self.seed = torch.tensor([seed], dtype=torch.int64, device="cuda")
        self.first = dict(weight=new(c, mean=1.0), gate=new(gates, c, mean=0.5), norm="rms", eps=1e-6, p=0.1, sequence=0)
        self.second = dict(weight=new(c, mean=1.0), bias=new(c), norm="layer", post_norm="rms", post_weight=new(c, mean=1.0),
                           eps=1e-5, p=0.25, sequence=1)
        self.wt, self.wts = t2s.quantize_fp8(self.w, along="columns", square=True)
        self.wn, self.wns = t2s.quantize_fp8(self.w, square=True)

    def forward(self, **kw):
        self.r, self.y = t2s.residual_norm(self.x, self.h, seed=self.seed, **self.first, **kw)
        self.yq, self.ys, self.yt, self.yts = t2s.quantize_fp8(self.y, along="both", **kw)
        self.z = t2s.gemm_fp8(self.yq, self.ys, self.wt.t(), self.wts.t(), dtype=self.dtype, **kw)
        self.r2, self.y2 = t2s.residual_norm(self.r, self.z, seed=self.seed, **self.second, **kw)
        self.out = t2s.dropout(self.y2, 0.1, self.seed, 2, residual=self.r2, **kw)

    def backward(self, **kw):
        self.dy2 = t2s.dropout_backward(self.dout, 0.1, self.seed, 2, **kw)
        self.g2 = t2s.residual_norm_backward(self.dy2, self.dout, self.r2, self.z, seed=self.seed, **self.second, **kw)
        self.dq, self.ds, self.dt, self.dts = t2s.quantize_fp8(self.g2.dh, dtype=E5M2, along="both", **kw)
        self.dy = t2s.gemm_fp8(self.dq, self.ds, self.wn.t(), self.wns.t(), dtype=self.dtype, **kw)
        self.dw = t2s.gemm_fp8(self.yt, self.yts, self.dt.t(), self.dts.t(), dtype=F32, **kw)
        self.g = t2s.residual_norm_backward(self.dy, self.g2.dx, self.r, self.h, seed=self.seed, **self.first, **kw)

    def run(self, **kw):
        self.forward(**kw)
        self.backward(**kw)

    def made(self):
        """Everything that a run made."""
        made = [self.r, self.y, self.yq, self.ys, self.yt, self.yts, self.z, self.r2, self.y2, self.out, self.dy2, *self.g2,
                self.dq, self.ds, self.dt, self.dts, self.dy, self.dw, *self.g]
        return [t for t in made if t is not None]

    def results(self):
        """Its bytes, copied."""
        return [t.flatten().clone(memory_format=torch.contiguous_format).view(torch.uint8) for t in self.made()]

    def check(self):
        seed, dtype = int(self.seed), self.dtype
        first, second = dict(self.first, seed=seed), dict(self.second, seed=seed)
        check_forward(first, self.x, self.h, self.r, self.y, dtype, "first")
        for got, scale, x, f8 in ((self.yq, self.ys, self.y, E4M3), (self.yt, self.yts, self.y.t(), E4M3),
                                  (self.dq, self.ds, self.g2.dh, E5M2), (self.dt, self.dts, self.g2.dh.t(), E5M2)):
            want, s = quantized(x, f8, False)
            assert bool((got.double() == want).all()) and bool((scale.double() == s).all())
        check_product(self.z, self.yq, self.ys, self.wt, self.wts, dtype, "z")
        check_forward(second, self.r, self.z, self.r2, self.y2, dtype, "second")
        keep = ref.factors(self.m, self.c, 0.1, seed, 2).cuda()
        part, r2 = self.y2.double() * keep, self.r2.double()
        within(self.out, part + r2, 2.0 ** -22 * (part.abs() + r2.abs()), dtype, "out")
        dy2 = self.dout.double() * keep
        within(self.dy2, dy2, 2.0 ** -22 * dy2.abs(), dtype, "dy2")
        check_backward(second, self.dy2, self.dout, self.r2, self.z, self.g2, dtype, "second")
        check_product(self.dy, self.dq, self.ds, self.wn, self.wns, dtype, "dy")
        check_product(self.dw, self.yt, self.yts, self.dt, self.dts, F32, "dw")
        check_backward(first, self.dy, self.g2.dx, self.r, self.h, self.g, dtype, "first")


def same(a, b):
    return len(a) == len(b) and all(s.shape == t.shape and bool((s == t).all()) for s, t in zip(a, b))


@pytest.mark.parametrize("m,c,dtype,gates", [(1, 512, BF16, 1), (12, 200, F16, 3), (300, 1001, BF16, 2), (1024, 640, F16, 4),
                                             (513, 2048, BF16, 1)])
def test_block(m, c, dtype, gates):
    block = Block(m, c, dtype, gates, m + c)
    block.run()
    block.check()
    assert binding.device_status() == binding.T2S_OK


def test_blocks_at_once():
    """Two blocks on two streams, call by call in turn, and as two graphs that are replayed at once: the bits of a run alone."""
    blocks = [Block(300, 1001, BF16, 2, 3), Block(777, 520, F16, 7, 4)]
    want = []
    for b in blocks:
        b.run()
        want.append(b.results())
    streams = [torch.cuda.Stream() for _ in blocks]
    torch.cuda.synchronize()
    for _ in range(3):
        for step in ("forward", "backward"):
            for b, s in zip(blocks, streams):
                with torch.cuda.stream(s):
                    getattr(b, step)()
    torch.cuda.synchronize()
    assert all(same(b.results(), w) for b, w in zip(blocks, want))
    graphs = []
    for b, s in zip(blocks, streams):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            b.run()
        graphs.append(graph)
    for _ in range(3):
        for t in (t for b in blocks for t in b.made()):
            t.view(torch.uint8).zero_() if t.element_size() == 1 else t.zero_()
        torch.cuda.synchronize()
        for _ in range(4):
            for graph, s in zip(graphs, streams):
                with torch.cuda.stream(s):
                    graph.replay()
        torch.cuda.synchronize()
    assert all(same(b.results(), w) for b, w in zip(blocks, want))
    for b, graph in zip(blocks, graphs):  # new masks, activations and gradients in place
        b.seed.add_(100)
        b.x.mul_(0.5)
        b.dout.neg_()
        graph.replay()
        torch.cuda.synchronize()
        b.check()
    assert binding.device_status() == binding.T2S_OK


def test_stream_argument():
    """The whole run with stream=, while torch's current stream is another one."""
    block = Block(129, 384, BF16, 3, 9)
    block.run()
    want = block.results()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    block.run(stream=side.cuda_stream)
    side.synchronize()
    assert same(block.results(), want)


def test_padded_batch():
    """Rows behind the last one of a batch neither change nor change anything; a batch of no rows."""
    m, c = 100, 640
    block = Block(m, c, BF16, 1, 5)
    block.run()
    want = block.results()
    wide = {}
    for name in ("x", "h", "dout"):
        wide[name] = torch.full((m + 60, c), float("nan"), dtype=BF16, device="cuda")
        wide[name][:m] = getattr(block, name)
        setattr(block, name, wide[name][:m])
    block.run()
    assert same(block.results(), want)
    assert all(bool(torch.isnan(t[m:]).all()) for t in wide.values())
    for name in ("x", "h", "dout"):
        setattr(block, name, wide[name][:0])
    block.run()
    assert block.out.shape == (0, c) and block.dy.shape == (0, c) and bool((block.dw == 0).all())
    assert all(bool((g == 0).all()) for g in (block.g.dweight, block.g.dgate, *(t for t in block.g2[2:] if t is not None)))


def test_scales_off_boundaries():
    """Scales at every offset within 16 bytes and at any strides: the bits of scales that lie together."""
    for m, k, n in ((3, 1000, 300), (300, 1000, 520), (70, 520, 257)):
        a, sa = operand(m, k, E4M3, 1, general=True)
        for square in (False, True):
            b, sb = operand(n, k, E5M2, 2, square=square, general=True)
            want = t2s.gemm_fp8(a, sa, b.t(), sb.t(), dtype=F32)
            for shift in range(4):
                def moved(s):
                    rows, cols = s.shape
                    frames = (torch.full((cols, rows + 4 - rows % 4 + 4 * (shift % 2)), float("nan"), device="cuda").t(),
                              torch.full((rows + 1, cols + 5), float("nan"), device="cuda"),
                              torch.full((2 * rows + 8, 3 * cols), float("nan"), device="cuda")[::2, ::3])
                    for f in frames:
                        v = f[shift:shift + rows, :cols] if shift + rows <= f.shape[0] else f[:rows, shift:shift + cols]
                        if v.shape == s.shape:
                            v.copy_(s)
                            yield v
                for va in moved(sa):
                    for vb in moved(sb):
                        assert bool((t2s.gemm_fp8(a, va, b.t(), vb.t(), dtype=F32) == want).all())
    assert binding.device_status() == binding.T2S_OK
