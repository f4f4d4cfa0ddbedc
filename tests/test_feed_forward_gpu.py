"""The feed-forward operators against their definitions in float64 (GPU tests).

Bars, element by element, with u the type's rounding (2^-8 bfloat16, 2^-11 float16) and t = 2^-24
half its smallest subnormal step (float16; 0 for bfloat16):
 - a sum of K products is off by at most K 2^-23 sum |a b| (every FP32 addition may truncate);
 - an activation's slope is at most 1.13 and its evaluation in FP32 is off by at most
   2^-17 (|z| + 1), a slope's by 2^-17 (|z| + 1);
 - an output is rounded once: u |y| + t;
 - dZ, dG and dU are rounded where they enter a product: u |dz| + t each.
"""
from __future__ import annotations

import math

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import roofline_driven_tiling_gb300 as t2s  # noqa: E402
from roofline_driven_tiling_gb300 import binding  # noqa: E402

BF16, F16 = torch.bfloat16, torch.float16
U = {BF16: 2.0 ** -8, F16: 2.0 ** -11}
TINY = {BF16: 0.0, F16: 2.0 ** -24}
ACTS = ["none", "relu", "silu", "gelu", "gelu_tanh"]
C, A = math.sqrt(2 / math.pi), 0.044715
CANARY = 77.0


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()
    torch.cuda.set_device(0)
    assert binding.device_status() == binding.T2S_OK


def act64(z, act):
    """act(z) and act'(z) in float64."""
    if act == "relu":
        return z.clamp(min=0), (z > 0).double()
    if act == "silu":
        s = torch.sigmoid(z)
        return z * s, s * (1 + z * (1 - s))
    if act == "gelu":
        p = torch.special.ndtr(z)
        return z * p, p + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    if act == "gelu_tanh":
        t = torch.tanh(C * (z + A * z ** 3))
        return z * (1 + t) / 2, (1 + t) / 2 + z * (1 - t * t) / 2 * C * (1 + 3 * A * z * z)
    return z, torch.ones_like(z)


class Maker:
    """Seeded tensors as views of larger ones: `pad` more columns per row and `shift` elements
    before the first; everything around a view holds a canary."""

    def __init__(self, seed, dtype, pad=0, shift=0):
        self.gen = torch.Generator(device="cuda").manual_seed(seed)
        self.dtype, self.pad, self.shift, self.frames = dtype, pad, shift, []

    def empty(self, rows, cols, pad=None):
        pad = self.pad if pad is None else pad
        ld = cols + pad
        frame = torch.full((rows * ld + self.shift + 64,), CANARY, dtype=self.dtype, device="cuda")
        view = frame[self.shift:self.shift + rows * ld].view(rows, ld)[:, :cols]
        self.frames.append((frame, view))
        return view

    def normal(self, rows, cols, scale=1.0):
        v = self.empty(rows, cols)
        v.copy_((torch.randn(rows, cols, generator=self.gen, device="cuda") * scale).to(self.dtype))
        return v

    def weight(self, k, n, wt):
        return self.normal(n, k, k ** -0.5 if k else 1.0).t() if wt else self.normal(k, n, k ** -0.5 if k else 1.0)

    def vector(self, n):
        return self.normal(1, n).reshape(n)

    def check_canaries(self):
        for frame, view in self.frames:
            view.fill_(CANARY)
            assert bool((frame == CANARY).all()), "write outside a matrix"


def within(got, want, bar, what):
    got = got.double()
    assert got.shape == want.shape
    assert bool(torch.isfinite(got).all()), what
    over = (got - want).abs() - bar
    worst = float(over.max()) if over.numel() else 0.0
    assert worst <= 0, "%s: %.3g over its bar" % (what, worst)


def linear_want(x, w, bias, residual, act, dtype):
    k = x.shape[1]
    x, w = x.double(), w.double()
    z = x @ w
    dz = (k + 2) * 2.0 ** -23 * (x.abs() @ w.abs())
    if bias is not None:
        z = z + bias.double()
        dz = dz + 2.0 ** -23 * z.abs()
    y = act64(z, act)[0]
    dy = 1.13 * dz + 2.0 ** -17 * (z.abs() + 1) * (act != "none")
    if residual is not None:
        y = y + residual.double()
        dy = dy + 2.0 ** -23 * y.abs()
    u, t = U[dtype], TINY[dtype]
    return y, dy * (1 + u) + u * y.abs() + t, z, dz * (1 + u) + u * z.abs() + t


def gated_want(x, wg, wu, act, dtype):
    """H and its bar, and (value, bar) of G and of U."""
    u, t = U[dtype], TINY[dtype]
    x, wg, wu = x.double(), wg.double(), wu.double()
    g, up, eps = x @ wg, x @ wu, (x.shape[1] + 2) * 2.0 ** -23
    dg, du = eps * (x.abs() @ wg.abs()), eps * (x.abs() @ wu.abs())
    value = act64(g, act)[0]
    dv = 1.13 * dg + 2.0 ** -17 * (g.abs() + 1)
    h = value * up
    bar = (dv * (up.abs() + du) + value.abs() * du + 2.0 ** -23 * h.abs()) * (1 + u) + u * h.abs() + t
    return h, bar, [(v, d * (1 + u) + u * v.abs() + t) for v, d in ((g, dg), (up, du))]


# Sizes around every tile edge (16, 32, 64, 128, 256), one value, one k step, odd everything.
SHAPES = [(1, 1, 1), (1, 64, 64), (1, 1024, 512), (2, 7, 5), (3, 264, 136), (15, 72, 1000), (16, 512, 256),
          (17, 513, 129), (31, 128, 4096), (33, 200, 328), (64, 1024, 192), (65, 96, 72), (100, 2048, 640),
          (127, 130, 126), (128, 128, 128), (129, 65, 257), (200, 777, 264), (256, 64, 512), (257, 320, 1016),
          (300, 64, 33), (511, 1032, 96), (640, 192, 2048), (1000, 997, 1003), (1025, 520, 776)]


@pytest.mark.parametrize("m,k,n", SHAPES)
def test_linear(m, k, n):
    for i, (dtype, wt) in enumerate([(BF16, False), (F16, True), (F16, False), (BF16, True)]):
        act, full = ACTS[(m + k + n + i) % 5], (m + i) % 2 == 0
        mk = Maker(100 + i, dtype)
        x, w = mk.normal(m, k), mk.weight(k, n, wt)
        bias = mk.vector(n) if full or i == 1 else None
        residual = mk.normal(m, n) if full else None
        out, preact = mk.empty(m, n), mk.empty(m, n) if i != 2 else None
        y, bar, z, zbar = linear_want(x, w, bias, residual, act, dtype)
        got = t2s.linear(x, w, bias, residual, act=act, out=out, preact=preact)
        assert got is out and binding.device_status() == binding.T2S_OK
        within(out, y, bar, "y %s %s wt=%s" % (act, dtype, wt))
        if preact is not None:
            within(preact, z, zbar, "z")
        mk.check_canaries()


@pytest.mark.parametrize("m,k,n", SHAPES)
def test_gated(m, k, n):
    for i, (dtype, wt) in enumerate([(BF16, False), (F16, True), (F16, False), (BF16, True)]):
        act = ACTS[(m + k + i) % 5]
        mk = Maker(200 + i, dtype)
        x, wg, wu = mk.normal(m, k), mk.weight(k, n, wt), mk.weight(k, n, wt)
        out = mk.empty(m, n)
        preact = (mk.empty(m, n), mk.empty(m, n)) if i % 2 == 0 else None
        h, bar, gates = gated_want(x, wg, wu, act, dtype)
        t2s.gated_linear(x, wg, wu, act=act, out=out, preact=preact)
        assert binding.device_status() == binding.T2S_OK
        within(out, h, bar, "h %s %s wt=%s" % (act, dtype, wt))
        if preact is not None:
            within(preact[0], *gates[0], "g")
            within(preact[1], *gates[1], "u")
        mk.check_canaries()


# Sizes that just fill the GPU with tiles of one width each (256, 224, 192, 128 and 64 sums a row), and
# widths that do not divide the outputs.
WIDTHS = [(2000, 1024, 2304), (2000, 1024, 2016), (2000, 1024, 1728), (2000, 1024, 1152), (2000, 512, 576),
          (3102, 1600, 448), (3102, 1600, 864), (2500, 1600, 288), (1800, 700, 1000), (4000, 320, 1504)]


@pytest.mark.parametrize("m,k,n", WIDTHS)
@pytest.mark.parametrize("wt", [False, True])
def test_tile_widths(m, k, n, wt):
    mk = Maker(21, BF16)
    x, w, wu, bias = mk.normal(m, k), mk.weight(k, n, wt), mk.weight(k, n, wt), mk.vector(n)
    out, g, u = mk.empty(m, n), mk.empty(m, n), mk.empty(m, n)
    y, bar, z, zbar = linear_want(x, w, bias, None, "silu", BF16)
    t2s.linear(x, w, bias, act="silu", out=out, preact=g)
    within(out, y, bar, "y")
    within(g, z, zbar, "z")
    h, bar, gates = gated_want(x, w, wu, "silu", BF16)
    t2s.gated_linear(x, w, wu, out=out, preact=(g, u))
    within(out, h, bar, "h")
    within(g, *gates[0], "g")
    within(u, *gates[1], "u")
    assert binding.device_status() == binding.T2S_OK
    mk.check_canaries()


def product_bar(da, a, b, dtype):
    """Bar of a @ b where a (float64) is off by da and enters the product rounded."""
    u, t = U[dtype], TINY[dtype]
    entering = da * (1 + u) + u * a.abs() + t
    want = a @ b
    off = entering @ b.abs() + (a.shape[1] + 2) * 2.0 ** -23 * ((a.abs() + entering) @ b.abs())
    return want, off * (1 + u) + u * want.abs() + t


def sum_bar(da, a, dtype):
    u, t = U[dtype], TINY[dtype]
    want = a.sum(0)
    off = da.sum(0) + (a.shape[0] + 2) * 2.0 ** -23 * a.abs().sum(0)
    return want, off * (1 + u) + u * want.abs() + t


@pytest.mark.parametrize("m,k,n", SHAPES)
def test_linear_backward(m, k, n):
    for i, (dtype, wt) in enumerate([(BF16, False), (F16, True), (F16, False), (BF16, True)]):
        act = ACTS[(k + n + i) % 5]
        mk = Maker(300 + i, dtype)
        dy, x, w, z = mk.normal(m, n), mk.normal(m, k), mk.weight(k, n, wt), mk.normal(m, n)
        dx, db = mk.empty(m, k), mk.empty(1, n).reshape(n)
        dw = mk.empty(n, k).t() if wt else mk.empty(k, n)
        slope = act64(z.double(), act)[1]
        d = dy.double() * slope
        off = 2.0 ** -17 * (z.double().abs() + 1) * dy.double().abs() * (act != "none")
        t2s.linear_backward(dy, x, w, z, act=act, dx=dx, dw=dw, db=db)
        assert binding.device_status() == binding.T2S_OK
        within(dx, *product_bar(off, d, w.double().t(), dtype), "dx %s" % act)
        want, bar = product_bar(off.t(), d.t(), x.double(), dtype)
        within(dw, want.t(), bar.t(), "dw %s" % act)
        within(db, *sum_bar(off, d, dtype), "db %s" % act)
        mk.check_canaries()


@pytest.mark.parametrize("m,k,n", SHAPES)
def test_gated_backward(m, k, n):
    for i, (dtype, wt) in enumerate([(BF16, False), (F16, True), (F16, False), (BF16, True)]):
        act = ACTS[(m + n + i) % 5]
        mk = Maker(400 + i, dtype)
        dh, x, g, up = mk.normal(m, n), mk.normal(m, k), mk.normal(m, n), mk.normal(m, n)
        wg, wu = mk.weight(k, n, wt), mk.weight(k, n, wt)
        dx = mk.empty(m, k)
        dwg, dwu = [mk.empty(n, k).t() if wt else mk.empty(k, n) for _ in range(2)]
        value, slope = act64(g.double(), act)
        dg, du = dh.double() * up.double() * slope, dh.double() * value
        off = 2.0 ** -17 * (g.double().abs() + 1) * dh.double().abs()
        og, ou = off * up.double().abs(), off
        t2s.gated_linear_backward(dh, x, wg, wu, (g, up), act=act, dx=dx, dw_gate=dwg, dw_up=dwu)
        assert binding.device_status() == binding.T2S_OK
        a, abar = product_bar(og, dg, wg.double().t(), dtype)
        b, bbar = product_bar(ou, du, wu.double().t(), dtype)
        # The two products are one sum: its rounding steps see both halves.
        both = 2 * n * 2.0 ** -23 * (dg.abs() @ wg.double().abs().t() + du.abs() @ wu.double().abs().t())
        within(dx, a + b, abar + bbar + both, "dx %s" % act)
        for got, o, d, name in ((dwg, og, dg, "dw_gate"), (dwu, ou, du, "dw_up")):
            want, bar = product_bar(o.t(), d.t(), x.double(), dtype)
            within(got, want.t(), bar.t(), "%s %s" % (name, act))
        mk.check_canaries()


@pytest.mark.parametrize("m,k,n,pad,shift", [
    (m, k, n, pad, shift) for m, k, n in [(1, 256, 136), (20, 72, 264), (300, 136, 200)]
    for pad, shift in [(8, 8), (24, 0), (3, 0), (0, 1), (5, 3)]] + [
    # Odd widths inside rows that are 16-byte aligned: what lies behind them is not theirs.
    (1, 253, 133, 3, 0), (20, 69, 261, 3, 8), (300, 133, 197, 3, 0), (45, 70, 262, 10, 0)])
def test_strides_and_offsets(m, k, n, pad, shift):
    """Views of larger tensors: rows that stay 16-byte aligned and rows that do not."""
    for wt in (False, True):
        mk = Maker(7, BF16, pad, shift)
        x, w, bias, residual = mk.normal(m, k), mk.weight(k, n, wt), mk.vector(n), mk.normal(m, n)
        out, preact = mk.empty(m, n), mk.empty(m, n)
        y, bar, z, zbar = linear_want(x, w, bias, residual, "silu", BF16)
        t2s.linear(x, w, bias, residual, act="silu", out=out, preact=preact)
        within(out, y, bar, "y")
        within(preact, z, zbar, "z")
        dy, dx, db = mk.normal(m, n), mk.empty(m, k), mk.empty(1, n).reshape(n)
        dw = mk.empty(n, k).t() if wt else mk.empty(k, n)
        t2s.linear_backward(dy, x, w, act="none", dx=dx, dw=dw, db=db)
        zero = torch.zeros(m, n, dtype=torch.float64, device="cuda")
        within(dx, *product_bar(zero, dy.double(), w.double().t(), BF16), "dx")
        want, wbar = product_bar(zero.t(), dy.double().t(), x.double(), BF16)
        within(dw, want.t(), wbar.t(), "dw")
        within(db, *sum_bar(zero, dy.double(), BF16), "db")
        w2, g, u = mk.weight(k, n, wt), mk.empty(m, n), mk.empty(m, n)
        t2s.gated_linear(x, w, w2, out=out, preact=(g, u))
        h, bar, gates = gated_want(x, w, w2, "silu", BF16)
        within(out, h, bar, "h")
        within(g, *gates[0], "g")
        within(u, *gates[1], "u")
        assert binding.device_status() == binding.T2S_OK
        mk.check_canaries()


def test_exact_where_sums_are_exact():
    """Small integers: every product and sum is exact, so the outputs are too."""
    gen = torch.Generator(device="cuda").manual_seed(3)

    def ints(rows, cols):
        return torch.randint(-2, 3, (rows, cols), generator=gen, device="cuda").to(F16)

    for m, k, n in [(1, 300, 520), (40, 320, 1048), (384, 256, 520), (777, 100, 513)]:
        x, w, w2, r = ints(m, k), ints(k, n), ints(k, n), ints(m, n)
        b = ints(1, n).reshape(n)
        z = x.double() @ w.double() + b.double()
        assert torch.equal(t2s.linear(x, w, b, r, act="relu").double(), z.clamp(min=0) + r.double())
        dx, dw, db = t2s.linear_backward(r, x, w, db=None)
        assert torch.equal(dx.double(), r.double() @ w.double().t())
        assert torch.equal(dw.double(), x.double().t() @ r.double())
        assert torch.equal(db.double(), r.double().sum(0))
        g, u = x.double() @ w.double(), x.double() @ w2.double()
        h = t2s.gated_linear(x, w, w2, act="relu").double()
        want = (g.clamp(min=0) * u)
        assert torch.equal(h, want.to(F16).double())


def test_lengths_of_zero():
    for dtype in (BF16, F16):
        mk = Maker(11, dtype)
        b, r = mk.vector(40), mk.normal(9, 40)
        x, w = mk.empty(9, 0), mk.empty(0, 40)
        y = t2s.linear(x, w, b, r, act="silu")
        want = act64(b.double(), "silu")[0] + r.double()
        within(y, want, (U[dtype] * want.abs() + 2.0 ** -16), "k = 0")
        assert t2s.linear(mk.empty(0, 8), mk.normal(8, 5)).shape == (0, 5)
        assert t2s.linear(mk.normal(4, 8), mk.empty(8, 0)).shape == (4, 0)
        assert bool((t2s.gated_linear(x, w, w) == 0).all())
        dx, dw, db = t2s.linear_backward(mk.empty(0, 40), mk.empty(0, 16), mk.normal(16, 40), mk.empty(0, 40),
                                         act="silu", db=None)
        assert dx.shape == (0, 16) and bool((dw == 0).all()) and bool((db == 0).all())
        dx, dw, db = t2s.linear_backward(mk.empty(6, 0), mk.normal(6, 16), mk.empty(16, 0), db=None)
        assert bool((dx == 0).all()) and dw.shape == (16, 0) and db.shape == (0,)
        dx, dg, du = t2s.gated_linear_backward(mk.empty(0, 40), mk.empty(0, 16), mk.normal(16, 40),
                                               mk.normal(16, 40), (mk.empty(0, 40), mk.empty(0, 40)))
        assert dx.shape == (0, 16) and bool((dg == 0).all()) and bool((du == 0).all())
        assert binding.device_status() == binding.T2S_OK


@pytest.mark.parametrize("m", [1, 24, 300])
def test_residual_in_place(m):
    k, n = 200, 776
    for dtype, n in ((BF16, 776), (F16, 777)):
        mk = Maker(5, dtype)
        x, w, r = mk.normal(m, k), mk.normal(k, n), mk.normal(m, n)
        want = t2s.linear(x, w, residual=r, act="gelu")
        got = t2s.linear(x, w, residual=r, act="gelu", out=r)
        assert got is r and torch.equal(got, want)


@pytest.mark.parametrize("m,k,n", [(1, 2048, 264), (48, 4096, 520), (700, 1000, 1304)])
def test_same_bits_every_time(m, k, n):
    mk = Maker(6, BF16)
    x, w, w2, dh = mk.normal(m, k), mk.normal(k, n), mk.normal(k, n), mk.normal(m, n)
    g, u = torch.empty_like(dh), torch.empty_like(dh)
    first = None
    for _ in range(5):
        now = [t2s.linear(x, w, act="gelu"), t2s.gated_linear(x, w, w2, preact=(g, u))]
        now += t2s.linear_backward(dh, x, w, g, act="silu", db=None)
        now += t2s.gated_linear_backward(dh, x, w, w2, (g, u))
        now = [v.clone() for v in now]
        if first is None:
            first = now
        assert all(torch.equal(a, b) for a, b in zip(first, now))


@pytest.mark.parametrize("m", [3, 300])
def test_values_outside_the_ordinary(m):
    """Infinities and NaN stay in the rows, columns and sums that they belong to."""
    k, n = 136, 264
    mk = Maker(8, BF16)
    x, w = mk.normal(m, k), mk.normal(k, n)
    clean = t2s.linear(x, w, act="gelu_tanh")
    xx = x.clone()
    xx[1, 5], xx[2, 7] = float("nan"), float("inf")
    y = t2s.linear(xx, w, act="gelu_tanh")
    assert bool(torch.isnan(y[1]).all())
    # +inf where the sum is +inf, -0 or NaN (inf * 0) where it is -inf.
    assert bool(torch.isinf(y[2][w[7] > 0]).all()) and not bool(torch.isposinf(y[2][w[7] < 0]).any())
    keep = [i for i in range(m) if i not in (1, 2)]
    assert torch.equal(y[keep], clean[keep])
    ww = w.clone()
    ww[3, 100] = float("nan")
    y = t2s.linear(x, ww, act="relu")
    assert bool(torch.isnan(y[:, 100]).all())
    others = [i for i in range(n) if i != 100]
    assert torch.equal(y[:, others], t2s.linear(x, w, act="relu")[:, others])
    # Far pre-activations: slopes are 0 and 1, nothing overflows into NaN.
    z = torch.full((m, n), 3e38, dtype=BF16, device="cuda")
    z[:, ::2] = -3e38
    for act in ("silu", "gelu", "gelu_tanh", "relu"):
        dy = torch.ones(m, n, dtype=BF16, device="cuda")
        _, _, db = t2s.linear_backward(dy, x, w, z, act=act, dx=False, dw=False, db=None)
        assert torch.equal(db.double(), torch.where(z[0] > 0, float(m), 0.0).double()), act
    assert binding.device_status() == binding.T2S_OK


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("m", [4, 140])
def test_gradients_against_differences(act, m):
    """Along a direction v, <gradient, v> is the slope of <dy, output> by central differences of
    the float64 definition; the bar sums the element bars along v."""
    k, n, h = 72, 136, 1e-5
    mk = Maker(9, F16)
    dtype = F16
    x, w, b, dy = mk.normal(m, k), mk.normal(k, n, k ** -0.5), mk.vector(n), mk.normal(m, n)
    z = torch.empty(m, n, dtype=dtype, device="cuda")
    t2s.linear(x, w, b, act=act, preact=z)
    if act == "relu":  # differences need every pre-activation away from the corner
        dy = torch.where(z.abs() > 0.01, dy, torch.zeros_like(dy))
    dx, dw, db = t2s.linear_backward(dy, x, w, z, act=act, db=None)
    X, W, B, D = x.double(), w.double(), b.double(), dy.double()

    def value(x, w, b):
        return float((D * act64(x @ w + b, act)[0]).sum())

    # The saved z is rounded: the slope moves by at most 1.2 per unit of z (its second derivative).
    zoff = 1.2 * (U[dtype] * z.double().abs() + 1e-3) * D.abs() + 2.0 ** -17 * (z.double().abs() + 1) * D.abs()
    if act in ("none", "relu"):
        zoff = 0 * zoff
    d = D * act64(z.double(), act)[1]
    gen = torch.Generator(device="cuda").manual_seed(1)
    for grad, at, bar in ((dx, 0, product_bar(zoff, d, W.t(), dtype)[1]),
                          (dw, 1, product_bar(zoff.t(), d.t(), X, dtype)[1].t()),
                          (db, 2, sum_bar(zoff, d, dtype)[1])):
        v = torch.randn(grad.shape, generator=gen, device="cuda", dtype=torch.float64)
        plus, minus = [[X, W, B], [X, W, B]]
        plus[at], minus[at] = plus[at] + h * v, minus[at] - h * v
        slope = (value(*plus) - value(*minus)) / (2 * h)
        assert abs(float((grad.double() * v).sum()) - slope) <= float((bar * v.abs()).sum()) + 1e-5 * abs(slope)
    # The gated pair, along its gate weight and its input.
    w2 = mk.normal(k, n, k ** -0.5)
    g, u = torch.empty_like(z), torch.empty_like(z)
    t2s.gated_linear(x, w, w2, act=act, preact=(g, u))
    if act == "relu":
        dy = torch.where(g.abs() > 0.01, dy, torch.zeros_like(dy))
    gx, gg, gu = t2s.gated_linear_backward(dy, x, w, w2, (g, u), act=act)
    D, W2 = dy.double(), w2.double()

    def gated_value(x, w, w2):
        return float((D * act64(x @ w, act)[0] * (x @ w2)).sum())

    G, S = g.double(), u.double()
    step = U[dtype] * (G.abs() + S.abs()) + 1e-3
    og = 2.4 * step * (S.abs() + 1) * D.abs()
    ou = 1.3 * step * D.abs()
    v1, s1 = act64(G, act)
    dg, du = D * S * s1, D * v1
    bars = (product_bar(og, dg, W.t(), dtype)[1] + product_bar(ou, du, W2.t(), dtype)[1],
            product_bar(og.t(), dg.t(), X, dtype)[1].t(), product_bar(ou.t(), du.t(), X, dtype)[1].t())
    for at, (grad, bar) in enumerate(zip((gx, gg, gu), bars)):
        v = torch.randn(grad.shape, generator=gen, device="cuda", dtype=torch.float64)
        plus, minus = [[X, W, W2], [X, W, W2]]
        plus[at], minus[at] = plus[at] + h * v, minus[at] - h * v
        slope = (gated_value(*plus) - gated_value(*minus)) / (2 * h)
        assert abs(float((grad.double() * v).sum()) - slope) <= float((bar * v.abs()).sum()) + 1e-5 * abs(slope)


def test_only_what_is_wanted():
    mk = Maker(12, BF16)
    dy, x, w, z = mk.normal(50, 64), mk.normal(50, 72), mk.normal(72, 64), mk.normal(50, 64)
    full = t2s.linear_backward(dy, x, w, z, act="silu", db=None)
    assert t2s.linear_backward(dy, x, w, z, act="silu", dx=False, dw=False) == (None, None, None)
    assert torch.equal(t2s.linear_backward(dy, x, w, z, act="silu", dw=False)[0], full[0])
    assert torch.equal(t2s.linear_backward(dy, x, w, z, act="silu", dx=False)[1], full[1])
    w2 = mk.normal(72, 64)
    gx, gg, gu = t2s.gated_linear_backward(dy, x, w, w2, (z, dy))
    assert torch.equal(t2s.gated_linear_backward(dy, x, w, w2, (z, dy), dw_gate=False, dw_up=False)[0], gx)
    assert torch.equal(t2s.gated_linear_backward(dy, x, w, w2, (z, dy), dx=False, dw_up=False)[1], gg)
    assert torch.equal(t2s.gated_linear_backward(dy, x, w, w2, (z, dy), dx=False, dw_gate=False)[2], gu)


def test_another_stream_and_a_graph():
    """On a stream that is not the current one, and replayed from a captured graph."""
    mk = Maker(13, F16)
    for m, n in ((4, 136), (300, 137)):
        x, w, w2, dh = mk.normal(m, 128), mk.normal(128, n), mk.normal(128, n), mk.normal(m, n)
        want = [t2s.gated_linear(x, w, w2), *t2s.linear_backward(dh, x, w, dh, act="gelu", db=None)]
        torch.cuda.synchronize()
        side = torch.cuda.Stream()
        got = [t2s.gated_linear(x, w, w2, stream=side.cuda_stream),
               *t2s.linear_backward(dh, x, w, dh, act="gelu", db=None, stream=side.cuda_stream)]
        side.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = [t2s.gated_linear(x, w, w2), *t2s.linear_backward(dh, x, w, dh, act="gelu", db=None)]
        for t in got:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_offsets_beyond_32_bits():
    """Matrices whose last rows lie more than 2^32 elements in."""
    m, k, n, ld = 66000, 24, 40, 65600
    dtype = BF16
    big_x = torch.empty(m, ld, dtype=dtype, device="cuda")
    big_y = torch.empty(m, ld, dtype=dtype, device="cuda")
    x, out = big_x[:, :k], big_y[:, :n]
    mk = Maker(14, dtype)
    x.copy_(mk.normal(m, k))
    w, b = mk.normal(k, n), mk.vector(n)
    t2s.linear(x, w, b, act="relu", out=out)
    want, bar, _, _ = linear_want(x, w, b, None, "relu", dtype)
    within(out, want, bar, "y")
    dx = big_x[:, 512:512 + k]
    dx, dw, db = t2s.linear_backward(out, x, w, dx=dx, db=None)
    zero = torch.zeros(m, n, dtype=torch.float64, device="cuda")
    within(dx, *product_bar(zero, out.double(), w.double().t(), dtype), "dx")
    want, wbar = product_bar(zero.t(), out.double().t(), x.double(), dtype)
    within(dw, want.t(), wbar.t(), "dw")
    within(db, *sum_bar(zero, out.double(), dtype), "db")


def test_refusals():
    mk = Maker(15, BF16)
    x, w, r = mk.normal(4, 16), mk.normal(16, 24), mk.normal(4, 24)
    with pytest.raises(TypeError):
        t2s.linear(x.float(), w)
    with pytest.raises(TypeError):
        t2s.linear(x, w.half())
    with pytest.raises(TypeError):
        t2s.linear(x.cpu(), w)
    with pytest.raises(TypeError):
        t2s.linear(x, w, residual=r.cpu())
    with pytest.raises(ValueError):
        t2s.linear(x, w, act="tanh")
    with pytest.raises(ValueError):
        t2s.linear(x, mk.normal(17, 24))
    with pytest.raises(ValueError):
        t2s.linear(x[:, ::2], w[:8])
    with pytest.raises(ValueError):
        t2s.linear(x[:1].expand(4, 16), w)
    with pytest.raises(ValueError):
        t2s.linear(x, w, bias=mk.vector(25))
    with pytest.raises(ValueError):
        t2s.linear(x, w, residual=mk.normal(4, 25))
    with pytest.raises(ValueError):
        t2s.linear_backward(r, x, w, act="silu")  # no pre-activations
    with pytest.raises(ValueError):
        t2s.linear_backward(r, mk.normal(5, 16), w)
    with pytest.raises(ValueError):
        t2s.gated_linear(x, w, mk.normal(24, 16).t())  # two orders
    with pytest.raises(t2s.binding.T2SError):
        t2s.linear(x, w, out=r, preact=r)
    with pytest.raises(t2s.binding.T2SError):
        t2s.linear_backward(r, x, w, r, act="silu", workspace=torch.empty(128, dtype=torch.uint8, device="cuda"))


@pytest.mark.parametrize("m,n", [(1 << 14, 1024), ((1 << 14) + 3, 1025), (1 << 21, 8), (6000, 4000),
                                 (40000, 44), (1 << 16, 64), (9000, 1000)])
def test_many_column_sums(m, n):
    """db of more values than a cluster's CTAs share."""
    mk = Maker(18, F16)
    dy, z, x, w = mk.normal(m, n), mk.normal(m, n), mk.normal(m, 16), mk.normal(16, n)
    dx, _, db = t2s.linear_backward(dy, x, w, z, act="silu", dw=False, db=None)
    d = dy.double() * act64(z.double(), "silu")[1]
    off = 2.0 ** -17 * (z.double().abs() + 1) * dy.double().abs()
    within(db, *sum_bar(off, d, F16), "db")
    within(dx, *product_bar(off, d, w.double().t(), F16), "dx")
    assert torch.equal(db, t2s.linear_backward(dy, x, w, z, act="silu", dx=False, dw=False, db=None)[2])


def test_many_rows():
    """More rows than a grid's second dimension has tiles, one output per row."""
    m, k, n = (1 << 24) + 1000, 8, 1
    mk = Maker(16, BF16)
    x, w, b = mk.normal(m, k), mk.normal(k, 8)[:, :n], mk.vector(n)
    y, bar, _, _ = linear_want(x, w, b, None, "relu", BF16)
    within(t2s.linear(x, w, b, act="relu"), y, bar, "y")
    dx, _, _ = t2s.linear_backward(x[:, :n], x, w, dw=False)
    zero = torch.zeros(m, n, dtype=torch.float64, device="cuda")
    within(dx, *product_bar(zero, x[:, :n].double(), w.double().t(), BF16), "dx")


def test_calls_on_several_streams_at_once():
    """Products of both kernels, gradients and the plain BF16 product side by side on four streams."""
    mk = Maker(17, BF16)
    a = [mk.normal(24, 2048), mk.normal(2048, 1536), mk.normal(2048, 1536), mk.normal(24, 1536)]
    b = [mk.normal(1200, 512), mk.normal(512, 2048), mk.normal(512, 2048), mk.normal(1200, 2048)]
    c = [mk.normal(640, 768), mk.normal(768, 640)]

    def gradients(x, w, w2, dh):
        return [*t2s.linear_backward(dh, x, w, dh, act="gelu", db=None),
                *t2s.gated_linear_backward(dh, x, w, w2, (dh, dh))]

    jobs = [lambda: [t2s.linear(a[0], a[1], act="silu"), t2s.gated_linear(*a[:3])],
            lambda: [t2s.linear(b[0], b[1], residual=b[3]), t2s.gated_linear(*b[:3])],
            lambda: gradients(*a) + gradients(*b), lambda: [t2s.gemm_bf16(*c)]]
    want = [job() for job in jobs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in jobs]
    got = [[] for _ in jobs]
    for _ in range(10):
        for i, (job, stream) in enumerate(zip(jobs, streams)):
            with torch.cuda.stream(stream):
                got[i].append(job())
    torch.cuda.synchronize()
    assert binding.device_status() == binding.T2S_OK
    for results, expected in zip(got, want):
        for result in results:
            assert all(torch.equal(r, e) for r, e in zip(result, expected))


@pytest.mark.parametrize("m,k,n,pad", [(1024, 64, 64, 0), (4096, 256, 256, 0), (4100, 264, 250, 6), (4100, 257, 131, 3),
                                       (16400, 768, 520, 0), (40001, 40, 1000, 8)])
def test_weight_gradients_over_many_rows(m, k, n, pad):
    """Rows enough that the weights' gradients are sums of several pieces."""
    for i, (dtype, wt) in enumerate([(BF16, False), (F16, True), (F16, False), (BF16, True)]):
        mk = Maker(500 + i, dtype, pad)
        dy, x, w, z, up = mk.normal(m, n), mk.normal(m, k), mk.weight(k, n, wt), mk.normal(m, n), mk.normal(m, n)
        dws = [mk.empty(n, k).t() if wt else mk.empty(k, n) for _ in range(5)]
        dx, db = mk.empty(m, k), mk.empty(1, n).reshape(n)
        value, slope = act64(z.double(), "silu")
        d, dl, du = dy.double() * slope, dy.double() * up.double() * slope, dy.double() * value
        off = 2.0 ** -17 * (z.double().abs() + 1) * dy.double().abs()
        ol = off * up.double().abs()
        t2s.linear_backward(dy, x, w, z, act="silu", dx=False, dw=dws[0], db=False)
        t2s.linear_backward(dy, x, w, z, act="silu", dx=dx, dw=dws[1], db=db)
        t2s.gated_linear_backward(dy, x, w, w, (z, up), act="silu", dx=False, dw_gate=dws[2], dw_up=False)
        t2s.gated_linear_backward(dy, x, w, w, (z, up), act="silu", dw_gate=dws[3], dw_up=dws[4])
        assert binding.device_status() == binding.T2S_OK
        within(dx, *product_bar(off, d, w.double().t(), dtype), "dx")
        within(db, *sum_bar(off, d, dtype), "db")
        for got, o, a, name in zip(dws, (off, off, ol, ol, off), (d, d, dl, dl, du),
                                   ("dw alone", "dw", "dw_gate alone", "dw_gate", "dw_up")):
            want, bar = product_bar(o.t(), a.t(), x.double(), dtype)
            within(got, want.t(), bar.t(), name)
        again = t2s.linear_backward(dy, x, w, z, act="silu", dx=False, dw=None, db=False)[1]
        assert torch.equal(again, dws[0])
        mk.check_canaries()
