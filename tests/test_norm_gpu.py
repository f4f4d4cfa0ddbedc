"""Norms with residual, gate and dropout, their gradients, and dropout, against float64 (GPU tests).

Bars, element by element: the bounds of norm_reference on FP32 statistics and sums, and one rounding of
the output: u |v| + t with u the type's half step (2^-8 bfloat16, 2^-11 float16) and t = 2^-25 half its
smallest subnormal step (float16; bfloat16's is below every value here).
"""
from __future__ import annotations

import math

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import norm_reference as ref  # noqa: E402
import roofline_driven_tiling_gb300 as t2s  # noqa: E402
from roofline_driven_tiling_gb300 import binding  # noqa: E402

BF16, F16 = torch.bfloat16, torch.float16
U, TINY = {BF16: 2.0 ** -8, F16: 2.0 ** -11}, {BF16: 0.0, F16: 2.0 ** -25}
CANARY = 77.0


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()
    torch.cuda.set_device(0)
    assert binding.device_status() == binding.T2S_OK


class Maker:
    """Seeded tensors as views of larger ones filled with a canary: `pad` more columns per row, `shift` elements
    before the first."""

    def __init__(self, seed, dtype, pad=0, shift=0):
        self.gen = torch.Generator(device="cuda").manual_seed(seed)
        self.dtype, self.pad, self.shift, self.frames = dtype, pad, shift, []

    def empty(self, rows, cols):
        ld = cols + self.pad
        frame = torch.full((rows * ld + self.shift + 64,), CANARY, dtype=self.dtype, device="cuda")
        view = frame[self.shift:self.shift + rows * ld].view(rows, ld)[:, :cols]
        self.frames.append((frame, view))
        return view

    def normal(self, rows, cols, scale=1.0, mean=0.0):
        v = self.empty(rows, cols)
        v.copy_((mean + torch.randn(rows, cols, generator=self.gen, device="cuda") * scale).to(self.dtype))
        return v

    def vector(self, n, mean=0.0):
        return (mean + 0.3 * torch.randn(n, generator=self.gen, device="cuda")).to(self.dtype)

    def check_canaries(self):
        for frame, view in self.frames:
            view.fill_(CANARY)
            assert bool((frame == CANARY).all()), "write outside a matrix"


def within(got, want, bar, dtype, what):
    got, bar = got.double(), bar * (1 + U[dtype]) + U[dtype] * want.abs() + TINY[dtype]
    assert got.shape == want.shape, what
    assert bool(torch.isfinite(got).all()), what
    over = (got - want).abs() - bar
    assert float(over.max()) <= 0 if over.numel() else True, "%s: %.3g over its bar" % (what, float(over.max()))


# Row lengths around every width of a thread's words, a warp, a block; beyond every fast kernel's limit.
SIZES = [(1, 1), (3, 2), (5, 7), (4, 8), (7, 31), (2, 32), (9, 64), (33, 100), (6, 255), (8, 256), (5, 257), (16, 512),
         (305, 520), (4, 777), (70, 1003), (12, 1024), (3, 1032), (40, 2048), (6, 2056), (5, 4095), (8, 4096), (3, 4104),
         (2, 5001), (6, 8192), (3, 8200), (2, 12288), (2, 16384), (2, 16392), (3, 20001), (700, 128), (1300, 72)]
NORMS = ["rms", "layer"]


def build(mk, i, m, n, h=True):
    """A case's options and tensors by its number."""
    opt = {"norm": NORMS[i % 2], "eps": 1e-5}
    t = {"x": mk.normal(m, n), "h": mk.normal(m, n, 1.5, 0.5) if h else None}
    if i % 3 != 1:
        opt["weight"] = mk.vector(n, 1.0)
    if i % 4 >= 2:
        opt["bias"] = mk.vector(n)
    if h:
        opt["post_norm"] = ["none", "rms", "layer"][(i // 2) % 3]
        if opt["post_norm"] != "none" and i % 5 != 3:
            opt["post_weight"] = mk.vector(n, 1.0)
        if opt["post_norm"] != "none" and i % 3 == 0:
            opt["post_bias"] = mk.vector(n)
        gates = [0, 1, m, 2][i % 4]
        if gates and m % gates == 0:
            opt["gate"] = mk.vector(n, 0.5) if gates == 1 else mk.normal(gates, n, 0.5, 0.5)
        opt["scale"] = [1.0, 0.75][i % 2]
        if i % 3 == 2:
            opt.update(p=[0.1, 0.5][i % 2], seed=i - 3, sequence=i)
    return opt, t


def reference(opt, m, n):
    keep = ref.factors(m, n, opt["p"], opt["seed"], opt["sequence"]).cuda() if "p" in opt else None
    return ref.Case(opt["norm"], opt.get("post_norm", "none"), opt["eps"], opt.get("scale", 1.0), keep,
                    **{k: opt[k] for k in ("weight", "bias", "gate", "post_weight", "post_bias") if k in opt})


def check_forward(opt, x, h, r, y, dtype, what):
    m, n = x.shape
    case, x64 = reference(opt, m, n), x.double()
    if h is None:
        assert r is x
        r64 = x64
    else:
        h64, gate = h.double(), ref.per_row(case.gate, m)
        branch = case.branch(h64)
        weight = 1.0 if case.post_weight is None else case.post_weight.abs()
        keep = 1.0 if case.keep is None else case.keep
        bar = ref.normed_error(h64, case.post, case.eps) * weight * keep if case.post != "none" else 0.0
        if case.post_bias is not None:
            bar = bar + 2.0 ** -22 * case.post_bias.abs() * keep
        bar = abs(gate) * (bar + 2.0 ** -22 * branch.abs()) + 2.0 ** -22 * (case.scale * x64).abs()
        within(r, case.stream(x64, h64), bar, dtype, what + " r")
        r64 = r.double()
    if opt["norm"] != "none":
        weight = 1.0 if case.weight is None else case.weight.abs()
        bar = ref.normed_error(r64, case.norm, case.eps) * weight
        bar = bar + 2.0 ** -22 * (0.0 if case.bias is None else case.bias.abs())
        within(y, case.y(r64), bar, dtype, what + " y")


def check_backward(opt, dy, dr, r, h, got, dtype, what):
    m, n = r.shape
    case = reference(opt, m, n)
    d64 = lambda t: None if t is None else t.double()  # noqa: E731
    want = case.gradients(d64(dy), d64(dr), r.double(), d64(h))
    r64, E, n_rows = r.double(), ref.E(n), m
    d_bar = 2.0 ** -22 * want["d"].abs()
    if dy is not None:
        g = dy.double() if case.weight is None else dy.double() * case.weight
        d_bar = d_bar + ref.through_error(g, r64, case.norm, case.eps)
        if dr is not None:
            d_bar = d_bar + 2.0 ** -22 * dr.double().abs()
    within(got.dx, want["dx"], abs(case.scale) * d_bar, dtype, what + " dx")
    rows_E = (n_rows + 16) * 2.0 ** -23  # a sum over all rows, one after another

    def total(name, t, term_bars, groups=1):
        if t is None:
            return
        w = want[name]
        bar = rows_E * want["|%s|" % name]
        if term_bars is not None:
            bar = bar + term_bars.view(groups, -1, n).sum(1)
        within(t.view(w.shape), w, bar, dtype, what + " " + name)

    if dy is not None:
        total("dweight", got.dweight, dy.double().abs() * ref.normed_error(r64, case.norm, case.eps))
        total("dbias", got.dbias, None)
    if h is None:
        return
    h64, gate = h.double(), ref.per_row(case.gate, m)
    gates = 1 if case.gate is None or case.gate.dim() == 1 else case.gate.shape[0]
    keep = 1.0 if case.keep is None else case.keep
    hh = ref.normed(h64, case.post, case.eps)[0]
    hh_bar = ref.normed_error(h64, case.post, case.eps) if case.post != "none" else torch.zeros_like(hh)
    weight = 1.0 if case.post_weight is None else case.post_weight.abs()
    branch = case.branch(h64)
    bias = 0.0 if case.post_bias is None else case.post_bias.abs()
    branch_bar = keep * (hh_bar * weight + 2.0 ** -22 * (hh.abs() * weight + bias))
    total("dgate", got.dgate, d_bar * branch.abs() + want["d"].abs() * branch_bar + 2.0 ** -22 * (want["d"] * branch).abs(),
          gates)
    dn, dn_bar = want["dn"], d_bar * abs(gate) * keep + 2.0 ** -22 * want["dn"].abs()
    total("dpost_weight", got.dpost_weight, dn_bar * hh.abs() + dn.abs() * hh_bar)
    total("dpost_bias", got.dpost_bias, dn_bar)
    q = dn if case.post_weight is None else dn * case.post_weight
    bar = ref.through_error(q, h64, case.post, case.eps)
    # The same map of an error of q: at most its own size and two means of it.
    inv = ref.normed(h64, case.post, case.eps)[1]
    qb = dn_bar * weight
    spread = qb if case.post == "none" else inv * (qb + qb.mean(1, keepdim=True) + hh.abs() * (qb * hh.abs()).mean(1, keepdim=True))
    within(got.dh, want["dh"], bar + spread, dtype, what + " dh")


@pytest.mark.parametrize("m,n", SIZES)
def test_forward_and_backward(m, n):
    for i, (dtype, pad, shift, h) in enumerate([(BF16, 0, 0, True), (F16, 0, 0, True), (F16, 3, 1, True), (BF16, 8, 8, True),
                                                (BF16, 5, 0, False), (F16, 0, 0, False)]):
        i += 3 * m + n
        mk = Maker(i, dtype, pad, shift)
        opt, t = build(mk, i, m, n, h)
        x, hh = t["x"], t["h"]
        r, y = (mk.empty(m, n) if h else None), mk.empty(m, n)
        got = t2s.residual_norm(x, hh, r=r, y=y, **opt)
        assert got[1] is y
        check_forward(opt, x, hh, got[0], y, dtype, str(opt.keys()))
        dy, dr = mk.normal(m, n), (mk.normal(m, n) if i % 4 else None)
        dx, dh = mk.empty(m, n), (mk.empty(m, n) if h else None)
        g = t2s.residual_norm_backward(dy, dr, got[0], hh, dx=dx, dh=dh, **opt)
        check_backward(opt, dy, dr, got[0], hh, g, dtype, str(opt.keys()))
        # The same bits again, and with outputs that the call allocates.
        again = t2s.residual_norm_backward(dy, dr, got[0], hh, **opt)
        for a, b in zip(g, again):
            assert a is b is None or bool((a == b).all())
        mk.check_canaries()
    assert binding.device_status() == binding.T2S_OK


@pytest.mark.parametrize("m,n", [(1, 4096), (9, 640), (33, 1001), (3, 9000), (2, 20000)])
def test_without_the_second_norm(m, n):
    """The residual stream alone: no y, no dy."""
    mk = Maker(5, BF16)
    x, h, gate = mk.normal(m, n), mk.normal(m, n), mk.vector(n, 0.5)
    opt = dict(norm="none", post_norm="rms", gate=gate, scale=0.5, eps=1e-6, p=0.2, seed=11, sequence=4)
    r, y = t2s.residual_norm(x, h, **opt)
    assert y is None
    check_forward(opt, x, h, r, y, BF16, "none")
    dr = mk.normal(m, n)
    check_backward(opt, None, dr, r, h, t2s.residual_norm_backward(None, dr, r, h, **opt), BF16, "none")


@pytest.mark.parametrize("gates,m", [(1, 2500), (2, 2500), (100, 300), (152, 304), (153, 306), (400, 400), (500, 1500), (1, 1)])
def test_gates(gates, m):
    """Every way in which the rows of the gates lie on the blocks."""
    n = 136
    for dtype in (BF16, F16):
        mk = Maker(gates + m, dtype)
        x, h = mk.normal(m, n), mk.normal(m, n)
        opt = dict(norm="rms", weight=mk.vector(n, 1.0), gate=mk.normal(gates, n, 0.5, 0.5), post_norm="layer",
                   post_weight=mk.vector(n, 1.0), post_bias=mk.vector(n), eps=1e-6)
        r, y = t2s.residual_norm(x, h, **opt)
        check_forward(opt, x, h, r, y, dtype, "gates")
        dy, dr = mk.normal(m, n), mk.normal(m, n)
        check_backward(opt, dy, dr, r, h, t2s.residual_norm_backward(dy, dr, r, h, **opt), dtype, "gates")


@pytest.mark.parametrize("m,n", [(4096, 96), (20000, 64), (3001, 1000), (1200, 4096), (900, 8192), (257, 9001)])
def test_sums_over_rows_are_exact(m, n):
    """Sums of small integers: every partial sum is exact in FP32, so dbias and dgate are the float64 sums, rounded
    once. No norm's statistics are in dgate: d is dr, n is h."""
    mk = Maker(m, F16)
    gen = torch.Generator(device="cuda").manual_seed(1)
    dr, h, dy = (torch.randint(-3, 4, (m, n), generator=gen, device="cuda").to(F16) for _ in range(3))
    for gates in (1, 4 if m % 4 == 0 else 1):
        gate = torch.ones(gates, n, dtype=F16, device="cuda")
        g = t2s.residual_norm_backward(None, dr, h, h, norm="none", gate=gate, scale=1.0)
        want = (dr.double() * h.double()).view(gates, -1, n).sum(1)
        assert bool((g.dgate.double() == want.to(F16).double()).all())
        assert bool((g.dx == dr).all()) and bool((g.dh == dr).all())
    g = t2s.residual_norm_backward(dy, None, h, None, bias=mk.vector(n), norm="layer", eps=1.0)
    assert bool((g.dbias.double() == dy.double().sum(0).to(F16).double()).all())


@pytest.mark.parametrize("n", [8, 640, 1001, 4096, 9000, 20000])
def test_rows_of_their_own(n):
    """A row of zeros, a constant row, infinities and NaN stay in their rows."""
    m = 12
    mk = Maker(n, BF16)
    x = mk.normal(m, n)
    x[1] = 0
    x[3] = 2.5
    x[5, n // 2] = math.inf
    x[7, n - 1] = math.nan
    x[9, 0] = -3.3e38
    for kind in NORMS:
        r, y = t2s.residual_norm(x, norm=kind, eps=1e-6)
        ok = [i for i in range(m) if i not in (5, 7, 9)]
        case = ref.Case(kind, eps=1e-6)
        bar = ref.normed_error(x[ok].double(), kind, 1e-6)
        within(y[ok], case.y(x[ok].double()), bar, BF16, kind)
        assert bool((y[1] == 0).all())
        assert bool(torch.isnan(y[7]).all()) and bool(torch.isnan(y[5]).any())
        dy = mk.normal(m, n)
        g = t2s.residual_norm_backward(dy, None, x, norm=kind, eps=1e-6)
        want = case.gradients(dy[ok].double(), None, x[ok].double(), None)
        bar = ref.through_error(dy[ok].double(), x[ok].double(), kind, 1e-6)
        within(g.dx[ok], want["dx"], bar, BF16, kind)
    # A dropped value is 0 whatever it was.
    h = torch.full((m, n), math.nan, dtype=BF16, device="cuda")
    keep = ref.factors(m, n, 0.5, 3, 1).cuda() != 0
    h[keep] = 1.0
    x = torch.ones(m, n, dtype=BF16, device="cuda")
    r, _ = t2s.residual_norm(x, h, norm="none", p=0.5, seed=3, sequence=1)
    assert bool((r.float() == torch.where(keep, 3.0, 1.0)).all())
    assert bool((t2s.residual_norm(x, h, norm="none", p=1.0)[0] == x).all())


@pytest.mark.parametrize("m,n", [(3, 1003), (40, 4096), (2, 17000)])
def test_in_place_and_streams(m, n):
    """r written over x; another stream; the same bits from a captured graph, and other masks when its seed moves."""
    mk = Maker(9, BF16)
    x, h, w = mk.normal(m, n), mk.normal(m, n), mk.vector(n, 1.0)
    seed = torch.tensor([5], dtype=torch.int64, device="cuda")
    opt = dict(weight=w, p=0.3, sequence=2, post_norm="rms", eps=1e-6)
    want = t2s.residual_norm(x, h, seed=5, **opt)
    into = x.clone()
    got = t2s.residual_norm(into, h, seed=seed, r=into, **opt)
    assert got[0] is into and bool((into == want[0]).all()) and bool((got[1] == want[1]).all())
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = t2s.residual_norm(x, h, seed=5, stream=side.cuda_stream, **opt)
    dy = mk.normal(m, n)
    side.synchronize()
    assert all(bool((a == b).all()) for a, b in zip(got, want))
    grads = t2s.residual_norm_backward(dy, None, want[0], h, seed=5, **opt)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        r, y = t2s.residual_norm(x, h, seed=seed, **opt)
        g = t2s.residual_norm_backward(dy, None, r, h, seed=seed, **opt)
    for value in (5, 6, 5):
        seed.fill_(value)
        graph.replay()
        torch.cuda.synchronize()
        assert bool((r == want[0]).all()) == (value == 5)
        if value == 5:
            assert bool((y == want[1]).all())
            assert all(a is b is None or bool((a == b).all()) for a, b in zip(g, grads))
    case = reference(dict(opt, norm="rms", seed=6), m, n)
    seed.fill_(6)
    graph.replay()
    bar = ref.normed_error(h.double(), "rms", 1e-6) * case.keep + 2.0 ** -22 * (case.branch(h.double()).abs() + x.double().abs())
    within(r, case.stream(x.double(), h.double()), bar, BF16, "replay")


@pytest.mark.parametrize("m,n", [(1, 1), (3, 5), (2, 8), (7, 64), (33, 1003), (129, 4096), (1000, 72), (5, 20001), (2, 70000)])
def test_dropout(m, n):
    for i, (dtype, pad, shift) in enumerate([(BF16, 0, 0), (F16, 3, 1), (BF16, 8, 8), (F16, 0, 0)]):
        mk = Maker(i, dtype, pad, shift)
        x, res = mk.normal(m, n), mk.normal(m, n)
        for p, seed, sequence in ((0.1, 3, 0), (0.5, -2, 7), (0.0, 1, 1), (1.0, 1, 1), (1e-5, 2 ** 63, 2 ** 62)):
            keep = ref.factors(m, n, p, seed, sequence).cuda()
            want = x.double() * keep
            y = t2s.dropout(x, p, seed, sequence, out=mk.empty(m, n))
            within(y, want, 2.0 ** -22 * want.abs(), dtype, "dropout")
            assert bool((y[keep == 0] == 0).all())
            g = t2s.dropout_backward(x, p, seed, sequence)
            assert bool((g == y).all())
            y = t2s.dropout(x, p, seed, sequence, residual=res, out=mk.empty(m, n))
            within(y, want + res.double(), 2.0 ** -22 * (want.abs() + res.double().abs()), dtype, "with residual")
            for target in (0, 1):  # over x, over the residual
                a, b = x.clone(), res.clone()
                assert bool((t2s.dropout(a, p, seed, sequence, residual=b, out=(a, b)[target]) == y).all())
        mk.check_canaries()
    x = torch.full((4, 50), math.inf, dtype=BF16, device="cuda")
    y = t2s.dropout(x, 0.5, 1)
    keep = ref.factors(4, 50, 0.5, 1, 0).cuda() != 0
    assert bool((y[~keep] == 0).all()) and bool(torch.isinf(y[keep]).all())


@pytest.mark.parametrize("n", [1, 3, 37, 1003, 2048])
@pytest.mark.parametrize("shift,pad", [(0, 0), (1, 4), (2, 3), (4, 8)])
def test_gate_gradients_of_any_stride(n, shift, pad):
    """The C entry point with dgate's rows at any place: the bits of rows on 16-byte boundaries, nothing written between them."""
    m = 6
    mk = Maker(n, BF16)
    dy, r, h, gate = mk.normal(m, n), mk.normal(m, n), mk.normal(m, n), mk.normal(m, n, 0.5, 0.5)
    want = t2s.residual_norm_backward(dy, None, r, h, gate=gate, eps=1e-6)
    frame = torch.full((m * (n + pad) + 16,), CANARY, dtype=BF16, device="cuda")
    dgate = frame[shift:shift + m * (n + pad)].view(m, n + pad)[:, :n]
    dx, dh = torch.empty_like(r), torch.empty_like(h)
    size = binding.t2s_residual_norm_backward_workspace_size(m, n, m, 1)
    workspace = torch.empty(size, dtype=torch.uint8, device="cuda")
    rc = binding.lib().t2s_residual_norm_backward_bf16(
        m, n, binding.T2S_NORM_RMS, binding.T2S_NORM_NONE, dy.data_ptr(), n, None, n, r.data_ptr(), n, h.data_ptr(), n, None,
        None, None, gate.data_ptr(), n, m, 1.0, 1e-6, 0, None, 0, 0, dx.data_ptr(), n, dh.data_ptr(), n, None, None, None,
        None, dgate.data_ptr(), n + pad, workspace.data_ptr(), size, torch.cuda.current_stream().cuda_stream)
    assert rc == binding.T2S_OK
    assert bool((dgate == want.dgate).all()) and bool((dx == want.dx).all()) and bool((dh == want.dh).all())
    dgate.fill_(CANARY)
    assert bool((frame == CANARY).all()), "write outside dgate"


def test_offsets_beyond_32_bits():
    """Rows whose offset passes 2^31 and 2^32 elements, from a tensor that spaces them so."""
    n, ld = 520, 1 << 28
    frame = torch.empty(17 * ld, dtype=BF16, device="cuda")
    x = frame.view(17, ld)[:, :n]
    x.copy_(torch.randn(17, n, device="cuda"))
    near = x.contiguous()
    h = torch.randn(17, n, device="cuda").to(BF16)
    opt = dict(p=0.2, seed=4, sequence=5, post_norm="rms")
    want = t2s.residual_norm(near, h, **opt)
    got = t2s.residual_norm(x, h, **opt)
    assert all(bool((a == b).all()) for a, b in zip(got, want))
    far = frame.view(17, ld)[:, 1024:1024 + n]
    far.copy_(want[0])
    a = t2s.residual_norm_backward(near, near, far, h, dx=x, **opt)
    b = t2s.residual_norm_backward(near, near, want[0], h, **opt)
    assert bool((a.dx == b.dx).all()) and bool((a.dh == b.dh).all())
    x.copy_(near)
    assert bool((t2s.dropout(x, 0.3, 1, out=x) == t2s.dropout(near, 0.3, 1)).all())


def test_refusals():
    mk = Maker(1, BF16)
    x, h, w = mk.normal(4, 64), mk.normal(4, 64), mk.vector(64)
    two = torch.zeros(2, dtype=torch.int64, device="cuda")
    for error, call in (
            (TypeError, lambda: t2s.residual_norm(x.float())), (TypeError, lambda: t2s.residual_norm(x, h.to(F16))),
            (TypeError, lambda: t2s.residual_norm(x, h.cpu())), (ValueError, lambda: t2s.residual_norm(x, h[:3])),
            (ValueError, lambda: t2s.residual_norm(x[0])), (ValueError, lambda: t2s.residual_norm(x.t())),
            (ValueError, lambda: t2s.residual_norm(x, weight=w[:63])), (ValueError, lambda: t2s.residual_norm(x, norm="l2")),
            (ValueError, lambda: t2s.residual_norm(x, gate=w)), (ValueError, lambda: t2s.residual_norm(x, p=0.1)),
            (ValueError, lambda: t2s.residual_norm(x, scale=2.0)), (ValueError, lambda: t2s.residual_norm(x, post_norm="rms")),
            (ValueError, lambda: t2s.residual_norm(x, norm="none")), (ValueError, lambda: t2s.residual_norm(x, r=h)),
            (ValueError, lambda: t2s.residual_norm(x, h, norm="none", weight=w)),
            (ValueError, lambda: t2s.residual_norm(x, h, norm="none", y=x)),
            (ValueError, lambda: t2s.residual_norm(x, h, post_weight=w)),
            (ValueError, lambda: t2s.residual_norm(x, h, gate=mk.normal(3, 64))),
            (ValueError, lambda: t2s.residual_norm(x, h, p=1.5)), (ValueError, lambda: t2s.residual_norm(x, h, seed=two)),
            (TypeError, lambda: t2s.residual_norm(x, h, seed=two[:1].int())),
            (binding.T2SError, lambda: t2s.residual_norm(x, h, r=h)), (binding.T2SError, lambda: t2s.residual_norm(x, h, y=x)),
            (binding.T2SError, lambda: t2s.residual_norm(x, h, eps=-1.0)),
            (ValueError, lambda: t2s.residual_norm_backward(None, x, x, h)),
            (ValueError, lambda: t2s.residual_norm_backward(x, x, h, norm="none")),
            (binding.T2SError, lambda: t2s.residual_norm_backward(x, x, h, dx=x)),
            (binding.T2SError, lambda: t2s.residual_norm_backward(x, None, h, weight=w, workspace=two)),
            (ValueError, lambda: t2s.dropout(x, -0.5)), (TypeError, lambda: t2s.dropout(x, 0.5, seed=0.5)),
            (TypeError, lambda: t2s.dropout(x.float(), 0.5)), (ValueError, lambda: t2s.dropout(x, 0.5, residual=h[:2])),
            (ValueError, lambda: t2s.residual_norm(x.clone().requires_grad_())),
            (ValueError, lambda: t2s.dropout(x.clone().requires_grad_(), 0.1))):
        with pytest.raises(error):
            call()
    with torch.no_grad():
        t2s.dropout(x.clone().requires_grad_(), 0.1)
    # Nothing to do, and sums over no rows.
    empty = torch.empty(0, 64, dtype=BF16, device="cuda")
    assert t2s.residual_norm(empty, empty, weight=w)[1].shape == (0, 64)
    g = t2s.residual_norm_backward(empty, None, empty, empty, weight=w, bias=w, gate=mk.normal(3, 64), post_norm="rms",
                                   post_weight=w, post_bias=w)
    assert all(bool((t == 0).all()) for t in g) and g.dgate.shape == (3, 64)
    assert t2s.dropout(empty, 0.5).shape == (0, 64)
    assert t2s.residual_norm(x[:, :0], h[:, :0])[1].shape == (4, 0)
    assert binding.device_status() == binding.T2S_OK
