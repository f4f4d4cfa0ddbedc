"""Products of 8-bit operands whose scales are far from one (GPU tests).

A block's sum may meet either scale first, or their product, but scales from 2^-94 to below 2^89 in magnitude take neither
out of FP32's normal range: bars are those of test_fp8_gpu, in both product kernels and with either kind of scales of b.
Outputs are FP32."""
from __future__ import annotations

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import roofline_driven_tiling_gb300 as t2s  # noqa: E402
from roofline_driven_tiling_gb300 import binding  # noqa: E402
from test_fp8_gpu import blocks, check_product, E4M3, E5M2, F32, operand  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()
    torch.cuda.set_device(0)
    assert binding.device_status() == binding.T2S_OK


# One tile of few rows, one of more, pairs of SMs in narrow and wide tiles, odd sizes.
@pytest.mark.parametrize("m,k,n", [(1, 4096, 1000), (3, 300, 128), (31, 1003, 999), (64, 640, 2048), (257, 1280, 1016),
                                   (640, 192, 2048), (2048, 512, 2048), (1000, 997, 1003)])
@pytest.mark.parametrize("square", [True, False])
def test_opposite_scales(m, k, n, square):
    """Scales of up to 2^88 against others of 2^-90 and the like, another pair for every block (operand's own are 2^-4 to 2^5)."""
    power = torch.tensor([83.0, -90.0, 0.0, 60.0, -83.0], device="cuda").repeat(blocks(k))[:blocks(k)]
    for general in (True, False):
        a, sa = operand(m, k, E4M3, m + n, general=general)
        b, sb = operand(n, k, E5M2, m + n + 1, square=square, general=general)
        sb[::3, ::2] = 0  # beside scales far from one, in their blocks
        for sign in (1, -1):
            far_a, far_b = sa * torch.exp2((sign * power).clamp(max=83)), sb * torch.exp2((-sign * power).clamp(max=83))
            c = t2s.gemm_fp8(a, far_a, b.t(), far_b.t(), dtype=F32)
            check_product(c, a, far_a, b, far_b, F32, "%s %d" % (general, sign))
    assert binding.device_status() == binding.T2S_OK


@pytest.mark.parametrize("m,k,n", [(16, 1024, 256), (512, 1024, 512)])
@pytest.mark.parametrize("square", [True, False])
def test_limits(m, k, n, square):
    """The largest sum there is, of either sign, times scales at both ends of their range and beside ones: powers of two, so that
    C is what a block's sum is with scales of one, times both, bit for bit."""
    for form, largest in ((E4M3, 448.0), (E5M2, 57344.0)):
        a = torch.full((m, k), largest, device="cuda").to(form)
        b = torch.full((n, k), largest, device="cuda").to(form)
        b[n // 2:] = (-b[n // 2:].float()).to(form)
        b[1::2] = torch.zeros(b[1::2].shape, device="cuda").to(form)
        b[1::2, 0] = torch.tensor(2.0 ** (-9 if form is E4M3 else -16), device="cuda").to(form)  # the least value, once
        groups = blocks(n) if square else n
        sa, sb = torch.zeros(m, blocks(k), device="cuda"), torch.zeros(groups, blocks(k), device="cuda")
        sa[:, 0], sb[:, 0] = 1.0, 1.0
        want = t2s.gemm_fp8(a, sa, b.t(), sb.t(), dtype=F32).double()  # the sums of the first block alone
        for x, y in ((88, -94), (-94, 88), (88, 0), (0, 88), (-94, 0), (0, -94)):
            sa[:, 0], sb[:, 0] = 2.0 ** x, 2.0 ** y
            c = t2s.gemm_fp8(a, sa, b.t(), sb.t(), dtype=F32)
            assert bool((c.double() == want * 2.0 ** (x + y)).all()), (form, x, y)
    assert binding.device_status() == binding.T2S_OK


@pytest.mark.parametrize("m,k,n", [(16, 1024, 256), (512, 1024, 512)])
@pytest.mark.parametrize("way", ["columns", "rows", "one column"])
def test_one_far_scale(m, k, n, way):
    """Scales far from one in one block leave every other row and column the bits that they had."""
    a, sa = operand(m, k, E4M3, 1)
    b, sb = operand(n, k, E4M3, 2)
    want = t2s.gemm_fp8(a, sa, b.t(), sb.t(), dtype=F32)
    far_a, far_b = sa.clone(), sb.clone()
    if way == "rows":
        far_a[5, 3] = 2.0 ** 80
    elif way == "columns":
        far_b[:, 3] *= 2.0 ** 80
        far_a[:, 3] *= 2.0 ** -80
    else:
        far_b[7, 3] = 2.0 ** -94
    c = t2s.gemm_fp8(a, far_a, b.t(), far_b.t(), dtype=F32)
    check_product(c, a, far_a, b, far_b, F32, way)
    rows, cols = torch.ones(m, dtype=torch.bool, device="cuda"), torch.ones(n, dtype=torch.bool, device="cuda")
    rows[5], cols[7] = way != "rows", way != "one column"
    assert bool((c[rows][:, cols] == want[rows][:, cols]).all())


def test_scales_below_the_range():
    """Blocks of zeros, whose scales are 2^-126, beside blocks of ordinary values: nothing is lost but what the header says."""
    gen = torch.Generator(device="cuda").manual_seed(3)
    for m, k, n in ((7, 600, 200), (300, 600, 520)):
        x = torch.randn(m, k, generator=gen, device="cuda")
        w = torch.randn(n, k, generator=gen, device="cuda")
        x[::2, 128:256], w[1::3, 256:384], x[1::4] = 0.0, 0.0, 2.0 ** -130
        a, sa = t2s.quantize_fp8(x)
        b, sb = t2s.quantize_fp8(w)
        assert float(sa.min()) == 2.0 ** -126 == float(sb.min())
        c = t2s.gemm_fp8(a, sa, b.t(), sb.t(), dtype=F32)
        check_product(c, a, sa, b, sb, F32, "zeros")
