"""What the 8-bit products, norms and dropout do with tensors that require grad (no GPU needed: CPU tensors stand for a
device's, and a call that passes its checks ends at the launch)."""
from __future__ import annotations

import pytest

torch = pytest.importorskip("torch")

from roofline_driven_tiling_gb300 import fp8  # noqa: E402
from test_fp8_norm_devices import device_zero, mat, turned  # noqa: E402, F401

E4M3, F32 = torch.float8_e4m3fn, torch.float32


def product_tensors():
    """a, its scales, b, its scales and the output, none of which requires grad."""
    return [mat(0, dtype=E4M3), mat(0, 4, 1, F32), turned(mat(0, dtype=E4M3)), turned(mat(0, 4, 1, F32)), mat(0, 4, 4)]


@pytest.mark.parametrize("which", range(4))
def test_product_refuses_inputs_that_require_grad(which):
    t = product_tensors()
    with pytest.raises(AssertionError, match="launched"):
        fp8.gemm_fp8(*t[:4], out=t[4])
    t[which].requires_grad_()
    with pytest.raises(ValueError, match="requires grad"):
        fp8.gemm_fp8(*t[:4], out=t[4])
    with torch.no_grad(), pytest.raises(AssertionError, match="launched"):
        fp8.gemm_fp8(*t[:4], out=t[4])


@pytest.mark.parametrize("which", (0, 2))
def test_product_refuses_casts_of_tensors_that_require_grad(which):
    """A cast to 8 bits, and views of it, keep the history of what was cast."""
    t = product_tensors()
    source = torch.randn(4, 128, requires_grad=True)
    cast = source.to(E4M3)
    assert cast.requires_grad
    cast = cast.as_subclass(type(t[0]))
    cast.index = 0
    t[which] = cast if which == 0 else turned(cast)
    with pytest.raises(ValueError, match="requires grad"):
        fp8.gemm_fp8(*t[:4], out=t[4])
    with torch.no_grad(), pytest.raises(AssertionError, match="launched"):
        fp8.gemm_fp8(*t[:4], out=t[4])
