"""8-bit values with a scale for each block of 128, and their products, against float64 (GPU tests).

quantize_fp8 is exact: x / scale is a quotient by a power of two, rounded once, so values and scales are
compared bit for bit. Bars of the product, element by element: with S the sum over blocks of the scaled
sum of a block's magnitudes, every addition within a block may truncate (128 2^-23 S = 2^-16 S), the
scales' product, the scaling and the additions over B blocks round ((B + 3) 2^-23 S, with one spare), and the output is
rounded once (u |c| + t).
"""
from __future__ import annotations

import math

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import roofline_driven_tiling_gb300 as t2s  # noqa: E402
from roofline_driven_tiling_gb300 import binding  # noqa: E402

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
E4M3, E5M2 = torch.float8_e4m3fn, torch.float8_e5m2
U, TINY = {BF16: 2.0 ** -8, F16: 2.0 ** -11, F32: 2.0 ** -24}, {BF16: 0.0, F16: 2.0 ** -25, F32: 2.0 ** -150}
LARGEST = {E4M3: 448.0, E5M2: 57344.0}


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()
    torch.cuda.set_device(0)
    assert binding.device_status() == binding.T2S_OK


def generator(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def blocks(n):
    return -(-n // 128)


def expand(scale, rows, cols):
    """Every value's scale."""
    s = scale.double().repeat_interleave(128, 1)[:, :cols]
    return s if s.shape[0] == rows else s.repeat_interleave(128, 0)[:rows]


def quantized(x, f8, square):
    """Values (as numbers) and scales, from the definition in float64."""
    m, n = x.shape
    x = x.double()
    wide = torch.zeros(blocks(m) * 128 if square else m, blocks(n) * 128, dtype=torch.float64, device=x.device)
    wide[:m, :n] = x.abs()
    amax = wide.view(-1, 128 if square else 1, blocks(n), 128).amax((1, 3))
    # The least power of two with amax <= largest * scale, counted down from far above.
    scale = torch.full_like(amax, 2.0 ** 127)
    for _ in range(127 + 126):
        half = scale / 2
        scale = torch.where(amax <= LARGEST[f8] * half, half, scale)
    q = x / expand(scale, m, n)
    # Nearest value, ties to even, over the type's sorted values.
    codes = torch.arange(256, dtype=torch.uint8, device=x.device).view(f8).double()
    values = codes[torch.isfinite(codes)].unique()
    at = torch.searchsorted(values, q).clamp(1, values.numel() - 1)
    low, high = values[at - 1], values[at]
    even = (torch.arange(values.numel(), device=x.device) - values.numel() // 2) % 2 == 0  # zero is even, codes alternate
    take_high = (q - low > high - q) | ((q - low == high - q) & even[at])
    return torch.where(take_high, high, low), scale


def operand(rows, k, f8, seed, square=False, pad=0, general=False):
    """8-bit rows with every exponent used, rows `pad` bytes further apart, and scales (general: not powers of
    two), with what they stand for."""
    gen = generator(seed)
    x = torch.randn(rows, k, generator=gen, device="cuda") * torch.exp2(torch.randint(-6, 3, (rows, k), generator=gen, device="cuda").float())
    frame = torch.full((rows, (k + 15) // 16 * 16 + pad), 0x7f, dtype=torch.uint8, device="cuda")  # NaN beyond the rows
    frame[:, :k] = x.clamp(-448, 448).to(f8).view(torch.uint8)
    q = frame.view(f8)[:, :k]
    groups = blocks(rows) if square else rows
    s = torch.exp2(torch.randint(-4, 5, (groups, blocks(k)), generator=gen, device="cuda").float())
    if general:
        s = s * (1 + torch.rand(groups, blocks(k), generator=gen, device="cuda"))
    return q, s


def check_product(c, a, sa, b, sb, dtype, what):
    (m, k), n = a.shape, b.shape[0]
    av, bv = a.double() * expand(sa, m, k), b.double() * expand(sb, n, k)
    want, size = av @ bv.t(), av.abs() @ bv.abs().t()
    bar = (128 + blocks(k) + 3) * 2.0 ** -23 * size
    bar = bar * (1 + U[dtype]) + U[dtype] * want.abs() + TINY[dtype]
    got = c.double()
    assert got.shape == want.shape and c.dtype is dtype
    assert bool(torch.isfinite(got).all()), what
    over = float(((got - want).abs() - bar).max())
    assert over <= 0, "%s: %.3g over its bar" % (what, over)


# Sizes around the widths of tiles and blocks; one value; long sums; few rows and many.
SHAPES = [(1, 1, 1), (1, 128, 128), (1, 4096, 1000), (2, 16, 7), (3, 129, 130), (8, 2048, 512), (15, 127, 257), (16, 256, 64),
          (17, 500, 129), (31, 1003, 999), (33, 384, 136), (48, 8192, 320), (64, 640, 2048), (65, 96, 72), (100, 2000, 640),
          (127, 130, 126), (128, 128, 128), (129, 65, 257), (200, 777, 264), (256, 512, 512), (257, 1280, 1016), (300, 64, 33),
          (511, 1032, 96), (640, 192, 2048), (1000, 997, 1003), (1025, 520, 776), (2049, 256, 1), (5, 20000, 40), (300, 33000, 200)]


@pytest.mark.parametrize("m,k,n", SHAPES)
def test_gemm(m, k, n):
    ways = [(E4M3, E4M3, BF16, True, False), (E4M3, E5M2, F32, False, True), (E5M2, E4M3, F16, True, True),
            (E5M2, E5M2, BF16, False, False), (E4M3, E4M3, F32, False, False)]
    for i, (fa, fb, dtype, square, general) in enumerate(ways):
        a, sa = operand(m, k, fa, 10 * i + m, pad=16 * (i % 2), general=general)
        b, sb = operand(n, k, fb, 10 * i + n + 1, square=square, pad=16 * (i % 3), general=general)
        sa = sa * 2.0 ** -6 / k ** 0.5  # binary16 outputs within range
        if i % 2:
            sa, sb = sa.t().contiguous().t(), sb.t().contiguous().t()
        c = t2s.gemm_fp8(a, sa, b.t(), sb.t(), dtype=dtype)
        check_product(c, a, sa, b, sb, dtype, str(ways[i]))
        assert bool((t2s.gemm_fp8(a, sa, b.t(), sb.t(), dtype=dtype) == c).all())
        frame = torch.full((m, n + 24), 77.0, dtype=dtype, device="cuda")
        shift = [8, 3, 1, 16, 2][i]
        out = frame[:, shift:shift + n]
        assert t2s.gemm_fp8(a, sa, b.t(), sb.t(), dtype=dtype, out=out) is out
        assert bool((out == c).all())
        out.fill_(77.0)
        assert bool((frame == 77.0).all()), "write outside the output"
    assert binding.device_status() == binding.T2S_OK


@pytest.mark.parametrize("m,k,n", [(1, 512, 300), (40, 1024, 257), (200, 2000, 384), (512, 640, 512), (700, 300, 500)])
def test_gemm_exact(m, k, n):
    """Small integers and scales of powers of two: every sum is exact, so C is the float64 result bit for bit."""
    gen = generator(m)
    for square in (True, False):
        a, b = (torch.randint(-4, 5, (r, (k + 15) // 16 * 16), generator=gen, device="cuda").float().to(E4M3)[:, :k] for r in (m, n))
        sa = torch.exp2(torch.randint(-2, 3, (m, blocks(k)), generator=gen, device="cuda").float())
        sb = torch.exp2(torch.randint(-2, 3, (blocks(n) if square else n, blocks(k)), generator=gen, device="cuda").float())
        want = (a.double() * expand(sa, m, k)) @ (b.double() * expand(sb, n, k)).t()
        c = t2s.gemm_fp8(a, sa, b.t(), sb.t(), dtype=F32)
        assert bool((c.double() == want).all())


def test_gemm_special_values():
    """Blocks of zeros, scales of zero, NaN and infinity stay in their rows and columns; no sum at all."""
    m, k, n = 70, 640, 300
    a, sa = operand(m, k, E4M3, 1)
    b, sb = operand(n, k, E4M3, 2)
    c = t2s.gemm_fp8(a, sa, b.t(), sb.t(), dtype=F32)
    sa2, sb2 = sa.clone(), sb.clone()
    sa2[3, 1], sa2[5, 4], sb2[7, 0] = math.nan, math.inf, math.nan
    sa2[6] = 0
    d = t2s.gemm_fp8(a, sa2, b.t(), sb2.t(), dtype=F32)
    rows, cols = torch.ones(m, dtype=torch.bool, device="cuda"), torch.ones(n, dtype=torch.bool, device="cuda")
    rows[[3, 5, 6]], cols[7] = False, False
    assert bool((d[rows][:, cols] == c[rows][:, cols]).all())
    assert bool(torch.isnan(d[3]).all()) and bool(torch.isnan(d[:, 7]).all())
    assert not bool(torch.isfinite(d[5]).any()) and bool((d[6][cols] == 0).all())
    one = torch.ones(1, 1, device="cuda")
    c = t2s.gemm_fp8(a, one.expand(m, 5), b.t(), one.expand(5, n), dtype=F32)  # one scale, repeated
    check_product(c, a, torch.ones(m, 5, device="cuda"), b, torch.ones(n, 5, device="cuda"), F32, "repeated")
    none = t2s.gemm_fp8(a[:, :0], sa[:, :0], b.t()[:0], sb.t()[:0])
    assert none.shape == (m, n) and bool((none == 0).all())
    assert t2s.gemm_fp8(a[:0], sa[:0], b.t(), sb.t()).shape == (0, n)
    assert t2s.gemm_fp8(a, sa, b.t()[:, :0], sb.t()[:, :0]).shape == (m, 0)


QSIZES = [(1, 1), (1, 128), (1, 4096), (2, 127), (3, 129), (16, 8), (17, 1000), (100, 100), (127, 384), (128, 128), (129, 257),
          (200, 2048), (333, 2800), (1000, 997), (700, 4100)]


@pytest.mark.parametrize("m,n", QSIZES)
def test_quantize(m, n):
    for i, (dtype, f8, square) in enumerate([(BF16, E4M3, False), (F16, E5M2, False), (F32, E4M3, False), (BF16, E5M2, True),
                                             (F32, E5M2, True), (F16, E4M3, True)]):
        gen = generator(m + n + i)
        pad = [0, 3, 0, 8, 1, 0][i]
        frame = torch.randn(m, n + pad, generator=gen, device="cuda")
        frame *= torch.exp2(torch.randint(-12, 4, (m, n + pad), generator=gen, device="cuda").float())
        x = frame.to(dtype)[:, :n]
        rows, columns = quantized(x, f8, square), quantized(x.t(), f8, square)
        for along, want in (("rows", rows), ("columns", columns), ("both", rows + columns)):
            got = t2s.quantize_fp8(x, dtype=f8, along=along, square=square)
            outs = []
            for g in got:  # the same into a caller's tensors, wider than they need be and off boundaries
                wide = torch.full((g.shape[0], g.shape[1] + 5), 1, dtype=torch.uint8 if g.dtype is f8 else F32, device="cuda")
                outs.append((wide, (wide.view(f8) if g.dtype is f8 else wide)[:, 2:2 + g.shape[1]]))
            again = t2s.quantize_fp8(x, dtype=f8, along=along, square=square, out=tuple(o for _, o in outs))
            assert len(got) == len(want)
            for g, w, o, (wide, view) in zip(got, want, again, outs):
                assert g.shape == w.shape and o is view
                assert bool((g.double() == w).all()) and bool((o.double() == w).all()), (along, dtype, f8, square)
                (view.view(torch.uint8) if g.dtype is f8 else view).fill_(1)
                assert bool((wide == 1).all()), "write outside an output"
    assert binding.device_status() == binding.T2S_OK


@pytest.mark.parametrize("f8", [E4M3, E5M2])
def test_quantize_values(f8):
    """Every value of the type and every midpoint, at the extremes of the scales; zeros; NaN and infinity."""
    codes = torch.arange(256, dtype=torch.uint8, device="cuda").view(f8).float()
    values = codes[torch.isfinite(codes)].unique()
    mid = (values[1:] + values[:-1]) / 2
    line = torch.cat([values, mid])
    line = torch.cat([line, torch.zeros(-line.numel() % 127, device="cuda")]).view(-1, 127)
    for power in (0, -40, 40, -100, 100, -126):
        x = torch.cat([torch.full((line.shape[0], 1), LARGEST[f8], device="cuda"), line], 1) * 2.0 ** power  # amax on the edge
        q, s = t2s.quantize_fp8(x, dtype=f8)
        w, ws = quantized(x, f8, False)
        assert bool((s.double() == ws).all()) and bool((s == 2.0 ** max(power, -126)).all()) and bool((q.double() == w).all()), power
        just_over = x.clone()
        just_over[:, 0] *= 1 + 2.0 ** -23
        assert bool((t2s.quantize_fp8(just_over, dtype=f8)[1] == 2.0 ** (power + 1)).all())
    tiny = torch.full((3, 200), 2.0 ** -149, device="cuda")
    tiny[1] = 0
    for along in ("rows", "columns"):
        q, s = t2s.quantize_fp8(tiny, dtype=f8, along=along)
        assert bool((s == 2.0 ** -126).all()) and bool((q.float() == 0).all())
    for dtype in (BF16, F16, F32):
        x = torch.randn(300, 300, generator=generator(1), device="cuda").to(dtype)
        clean = t2s.quantize_fp8(x, dtype=f8, along="both")
        x[5, 200], x[200, 7] = math.nan, -math.inf
        q, s, qt, st = t2s.quantize_fp8(x, dtype=f8, along="both")
        for got, scale, old, spots in ((q, s, clean, ((5, 1), (200, 0))), (qt, st, clean[2:], ((200, 0), (7, 1)))):
            bad = torch.zeros_like(scale, dtype=torch.bool)
            for r, b in spots:
                bad[r, b] = True
            assert bool((torch.isnan(scale) == bad).all()) and bool((scale[~bad] == old[1][~bad]).all())
            every = bad.repeat_interleave(128, 1)[:, :300]
            assert bool((torch.isnan(got.float()) == every).all())
            assert bool((got.float()[~every] == old[0].float()[~every]).all())
        q, s = t2s.quantize_fp8(x, dtype=f8, square=True)
        assert bool(torch.isnan(s).any()) and bool((torch.isnan(q.float()) == torch.isnan(expand(s, 300, 300))).all())


def test_linear_layer_and_its_gradients():
    """quantize_fp8 and gemm_fp8 as a layer uses them, forward and backward, on odd sizes."""
    m, k, n = 333, 300, 257
    gen = generator(4)
    x, dy = (torch.randn(m, c, generator=gen, device="cuda").to(BF16) for c in (k, n))
    w = torch.randn(k, n, generator=gen, device="cuda") * k ** -0.5
    wt, wts = t2s.quantize_fp8(w, along="columns", square=True)
    wn, wns = t2s.quantize_fp8(w, square=True)
    assert bool((wt.t().float() == wn.float()).all()) and bool((wts.t() == wns).all())
    xq, xs = t2s.quantize_fp8(x)
    check_product(t2s.gemm_fp8(xq, xs, wt.t(), wts.t()), xq, xs, wt, wts, BF16, "y")
    dq, ds, dt, dts = t2s.quantize_fp8(dy, dtype=E5M2, along="both")
    check_product(t2s.gemm_fp8(dq, ds, wn.t(), wns.t()), dq, ds, wn, wns, BF16, "dx")
    xt, xts = t2s.quantize_fp8(x, along="columns")
    dw = t2s.gemm_fp8(xt, xts, dt.t(), dts.t(), dtype=F32)
    check_product(dw, xt, xts, dt, dts, F32, "dw")
    # e5m2 rounds by up to 2^-3, e4m3 by 2^-4 of a value (more below its smallest normal value, 2^-9 of a scale
    # that is at most 2^-7.8 of a block's largest): the product of both against the unrounded one.
    want, size = x.double().t() @ dy.double(), x.double().abs().t() @ dy.double().abs()
    assert bool(((dw.double() - want).abs() <= 0.2 * size + 1e-3 * m).all())


def test_streams_and_graphs():
    m, k, n = 100, 1000, 520
    a, sa = operand(m, k, E4M3, 1)
    b, sb = operand(n, k, E4M3, 2, square=True)
    x = torch.randn(m, k, generator=generator(3), device="cuda").to(BF16)
    want, q = t2s.gemm_fp8(a, sa, b.t(), sb.t()), t2s.quantize_fp8(x, along="both")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    c, p = t2s.gemm_fp8(a, sa, b.t(), sb.t(), stream=side.cuda_stream), t2s.quantize_fp8(x, along="both", stream=side.cuda_stream)
    side.synchronize()
    assert bool((c == want).all()) and all(bool((s.float() == t.float()).all()) for s, t in zip(p, q))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        xq, xs = t2s.quantize_fp8(x)
        y = t2s.gemm_fp8(xq, xs, b.t(), sb.t())
    x.neg_()
    graph.replay()
    torch.cuda.synchronize()
    assert bool((xq.float() == -q[0].float()).all()) and bool((xs == q[1]).all())
    check_product(y, xq, xs, b, sb, BF16, "replayed")


def test_offsets_beyond_32_bits():
    """Rows beyond 2^31 and 2^32 bytes."""
    m, k, n, ld = 20, 300, 140, 1 << 28
    a, sa = operand(m, k, E4M3, 1)
    b, sb = operand(n, k, E4M3, 2)
    want = t2s.gemm_fp8(a, sa, b.t(), sb.t())
    far = torch.zeros(m * ld, dtype=torch.uint8, device="cuda").view(m, ld)
    far[:, :k] = a.view(torch.uint8)
    assert bool((t2s.gemm_fp8(far.view(E4M3)[:, :k], sa, b.t(), sb.t()) == want).all())
    x = torch.randn(m, k, generator=generator(5), device="cuda").to(BF16)
    q, s = t2s.quantize_fp8(x)
    spread = far.view(BF16)[:, 1024:1024 + k]
    spread.copy_(x)
    out = (far.view(E4M3)[:, :k], torch.empty_like(s))
    t2s.quantize_fp8(spread, out=out)
    assert bool((out[0].float() == q.float()).all()) and bool((out[1] == s).all())
    c = far.view(BF16)[:, 4096:4096 + n]
    t2s.gemm_fp8(a, sa, b.t(), sb.t(), out=c)
    assert bool((c == want).all())


def test_refusals():
    a, sa = operand(8, 256, E4M3, 1)
    b, sb = operand(300, 256, E4M3, 2)
    x = torch.zeros(8, 256, dtype=BF16, device="cuda")
    for error, call in (
            (TypeError, lambda: t2s.gemm_fp8(x, sa, b.t(), sb.t())), (TypeError, lambda: t2s.gemm_fp8(a, sa, x.t(), sb.t())),
            (TypeError, lambda: t2s.gemm_fp8(a, sa.half(), b.t(), sb.t())), (TypeError, lambda: t2s.gemm_fp8(a, sa, b.t(), sb.t().cpu())),
            (ValueError, lambda: t2s.gemm_fp8(a, sa, b, sb.t())), (ValueError, lambda: t2s.gemm_fp8(a, sa[:, :1], b.t(), sb.t())),
            (ValueError, lambda: t2s.gemm_fp8(a, sa, b.t(), sb.t()[:, :5])), (ValueError, lambda: t2s.gemm_fp8(a, sa, b.t(), sb)),
            (ValueError, lambda: t2s.gemm_fp8(a[:, 8:248], sa, b.t()[8:248], sb.t())),
            (ValueError, lambda: t2s.gemm_fp8(a, sa, b.t().contiguous(), sb.t())),
            (ValueError, lambda: t2s.gemm_fp8(a, sa, b.t(), sb.t(), dtype=torch.float64)),
            (TypeError, lambda: t2s.gemm_fp8(a, sa, b.t(), sb.t(), out=torch.empty(8, 300, device="cuda"))),
            (ValueError, lambda: t2s.gemm_fp8(a, sa, b.t(), sb.t(), out=torch.empty(8, 299, dtype=BF16, device="cuda"))),
            (ValueError, lambda: t2s.gemm_fp8(a, sa.clone().requires_grad_(), b.t(), sb.t())),
            (ValueError, lambda: t2s.quantize_fp8(x, dtype=torch.int8)), (ValueError, lambda: t2s.quantize_fp8(x, along="k")),
            (ValueError, lambda: t2s.quantize_fp8(x[0])), (ValueError, lambda: t2s.quantize_fp8(x.t())),
            (ValueError, lambda: t2s.quantize_fp8(x.clone().requires_grad_())),
            (ValueError, lambda: t2s.quantize_fp8(x, out=(a,))), (TypeError, lambda: t2s.quantize_fp8(x, out=(a, sa.half()))),
            (TypeError, lambda: t2s.quantize_fp8(x, dtype=E5M2, out=(a, sa))), (ValueError, lambda: t2s.quantize_fp8(x, out=(a, sa.t()))),
            (ValueError, lambda: t2s.quantize_fp8(x, out=(a[:, :255], sa))),
            (binding.T2SError, lambda: t2s.quantize_fp8(x, out=(a, sa[:1, :1].expand(8, 2))))):
        with pytest.raises(error):
            call()
    assert binding.device_status() == binding.T2S_OK
