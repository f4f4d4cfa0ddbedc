"""The 8-bit products' and norms' refusals of tensors on another device than their own (no GPU needed)."""
from __future__ import annotations

import pytest

torch = pytest.importorskip("torch")

from roofline_driven_tiling_gb300 import feed_forward, fp8, norm  # noqa: E402
import test_feed_forward_arguments as arguments  # noqa: E402

BF16, E4M3 = torch.bfloat16, torch.float8_e4m3fn


class Placed(arguments.OnDevice):
    device = property(lambda self: torch.device("cuda", self.index))


def on_device(index, shape=(4096,), dtype=torch.uint8):
    t = torch.empty(shape, dtype=dtype).as_subclass(Placed)
    t.index = index
    return t


@pytest.fixture(autouse=True)
def device_zero(monkeypatch):
    """Every check comes before anything is launched: no entry point of the library is reached."""
    monkeypatch.setattr(feed_forward, "_current_device", lambda: 0)
    monkeypatch.setattr(fp8, "_current_device", lambda: 0)

    def launch(*a):
        raise AssertionError("launched")
    monkeypatch.setattr(norm, "_function", lambda *a: launch)
    monkeypatch.setattr(fp8, "_function", lambda *a: launch)
    for module in (norm, fp8):
        monkeypatch.setattr(module, "_FUNCTIONS", {})
        monkeypatch.setattr(module, "_raw_stream", lambda index: 0)


def mat(index, rows=4, cols=128, dtype=BF16):
    return on_device(index, (rows, cols), dtype)


def turned(t):
    """Its transpose, on the same device."""
    out = t.t()
    out.index = t.index
    return out


def vec(index, n=128):
    return on_device(index, (n,), BF16)


def test_all_on_the_current_device():
    """The same calls with every tensor at home get as far as the launch."""
    x, h, r, y = (mat(0) for _ in range(4))
    for call in (lambda: norm.residual_norm(x, h, vec(0), gate=vec(0), p=0.1, seed=on_device(0, (1,), torch.int64), r=r, y=y),
                 lambda: norm.dropout(x, 0.5, residual=h, out=y),
                 lambda: norm.residual_norm_backward(y, r, x, h, dx=mat(0), dh=mat(0), workspace=on_device(0)),
                 lambda: fp8.quantize_fp8(x, out=(mat(0, dtype=E4M3), mat(0, 4, 1, torch.float32))),
                 lambda: fp8.gemm_fp8(mat(0, dtype=E4M3), mat(0, 4, 1, torch.float32), mat(0, dtype=E4M3).t(),
                                      mat(0, 1, 4, torch.float32), out=mat(0, 4, 4))):
        with pytest.raises(AssertionError, match="launched"):
            call()


def test_tensors_on_another_device():
    x, h, r, y, w = mat(0), mat(0), mat(0), mat(0), vec(0)
    far, line, seed = mat(1), vec(1), on_device(1, (1,), torch.int64)
    for call in (
            lambda: norm.residual_norm(far, h), lambda: norm.residual_norm(x, far), lambda: norm.residual_norm(x, h, line),
            lambda: norm.residual_norm(x, h, w, line), lambda: norm.residual_norm(x, h, gate=line),
            lambda: norm.residual_norm(x, h, gate=far), lambda: norm.residual_norm(x, h, post_norm="rms", post_weight=line),
            lambda: norm.residual_norm(x, h, post_norm="rms", post_bias=line), lambda: norm.residual_norm(x, h, r=far, y=y),
            lambda: norm.residual_norm(x, h, r=r, y=far), lambda: norm.residual_norm(x, h, p=0.1, seed=seed, r=r, y=y),
            lambda: norm.dropout(far, 0.1), lambda: norm.dropout(x, 0.1, residual=far), lambda: norm.dropout(x, 0.1, out=far),
            lambda: norm.dropout(x, 0.1, seed=seed, out=y), lambda: norm.dropout_backward(x, 0.1, dx=far),
            lambda: norm.residual_norm_backward(far, None, r, h), lambda: norm.residual_norm_backward(y, far, r, h),
            lambda: norm.residual_norm_backward(y, None, far, h), lambda: norm.residual_norm_backward(y, None, r, far),
            lambda: norm.residual_norm_backward(y, None, r, h, line), lambda: norm.residual_norm_backward(y, None, r, h, w, line),
            lambda: norm.residual_norm_backward(y, None, r, h, gate=line),
            lambda: norm.residual_norm_backward(y, None, r, h, dx=far),
            lambda: norm.residual_norm_backward(y, None, r, h, dx=x, dh=far),
            lambda: norm.residual_norm_backward(y, None, r, h, dx=x, dh=h, workspace=on_device(1))):
        with pytest.raises(ValueError):
            call()


def test_quantized_tensors_on_another_device():
    a, sa, b, sb = mat(0, dtype=E4M3), mat(0, 4, 1, torch.float32), mat(0, dtype=E4M3).t(), mat(0, 1, 4, torch.float32)
    far8, far_s, out = mat(1, dtype=E4M3), mat(1, 4, 1, torch.float32), mat(0, 4, 4)
    for call in (lambda: fp8.quantize_fp8(mat(1)), lambda: fp8.quantize_fp8(mat(0), out=(far8, sa)),
                 lambda: fp8.quantize_fp8(mat(0), out=(a, far_s)), lambda: fp8.gemm_fp8(far8, far_s, turned(far8), turned(far_s)),
                 lambda: fp8.gemm_fp8(a, far_s, b, sb, out=out), lambda: fp8.gemm_fp8(a, sa, turned(far8), sb, out=out),
                 lambda: fp8.gemm_fp8(a, sa, b, turned(far_s), out=out), lambda: fp8.gemm_fp8(a, sa, b, sb, out=mat(1, 4, 4))):
        with pytest.raises((ValueError, TypeError)):
            call()
