"""Gradients of parameters that are absent (all ones, zeros), which the C entry points give and the torch ones do not ask
for, against the same call with the ones and zeros in memory (GPU tests): dx and dh have its bits. Sums over rows need not,
since a block's shared memory, and with it the number of blocks that share the rows, depends on which arguments are there;
their bars are those of test_norm_gpu against float64."""
from __future__ import annotations

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import roofline_driven_tiling_gb300 as t2s  # noqa: E402
from roofline_driven_tiling_gb300 import binding, norm  # noqa: E402
from test_norm_gpu import check_backward  # noqa: E402

SUFFIX = {torch.bfloat16: "bf16", torch.float16: "f16"}


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()
    torch.cuda.set_device(0)
    assert binding.device_status() == binding.T2S_OK


@pytest.mark.parametrize("m,n,gates", [(6, 64, 1), (60, 520, 3), (300, 72, 100), (400, 1003, 400), (35, 4097, 7), (9, 9001, 3)])
@pytest.mark.parametrize("kind,post", [("layer", "rms"), ("rms", "layer")])
def test_gradients_of_absent_parameters(m, n, gates, kind, post):
    dtype = torch.bfloat16 if m % 2 else torch.float16
    gen = torch.Generator(device="cuda").manual_seed(m + n)
    dy, dr, r, h = (torch.randn(m, n, generator=gen, device="cuda").to(dtype) for _ in range(4))
    one, zero = torch.ones(n, dtype=dtype, device="cuda"), torch.zeros(n, dtype=dtype, device="cuda")
    opt = dict(weight=one, bias=zero, gate=torch.ones(gates, n, dtype=dtype, device="cuda"), norm=kind, post_norm=post,
               post_weight=one, post_bias=zero, scale=0.5, eps=1e-5, p=0.2, seed=7, sequence=1)
    want = t2s.residual_norm_backward(dy, dr, r, h, **opt)
    check_backward(opt, dy, dr, r, h, want, dtype, "with ones")
    new = lambda rows: torch.full((rows, n), 77.0, dtype=dtype, device="cuda")  # noqa: E731
    names = ("dweight", "dbias", "dpost_weight", "dpost_bias", "dgate")
    for wanted in (names, ("dgate",), ("dbias", "dpost_weight"), ()):
        out = {name: new(gates if name == "dgate" else 1) for name in wanted}
        dx, dh = new(m), new(m)
        size = binding.t2s_residual_norm_backward_workspace_size(m, n, gates, len(wanted))
        workspace = torch.empty(max(size, 1), dtype=torch.uint8, device="cuda")
        at = [out[name].data_ptr() if name in out else None for name in names]
        rc = getattr(binding.lib(), "t2s_residual_norm_backward_" + SUFFIX[dtype])(
            m, n, norm.NORMS[kind], norm.NORMS[post], dy.data_ptr(), n, dr.data_ptr(), n, r.data_ptr(), n, h.data_ptr(), n, None,
            None, None, None, n, gates, 0.5, 1e-5, norm._dropped(0.2), None, 7, 1, dx.data_ptr(), n, dh.data_ptr(), n, *at, n,
            workspace.data_ptr(), size, torch.cuda.current_stream().cuda_stream)
        assert rc == binding.T2S_OK
        assert bool((dx == want.dx).all()) and bool((dh == want.dh).all())
        got = want._replace(dx=dx, dh=dh, **{name: v if name == "dgate" else v[0] for name, v in out.items()})
        check_backward(opt, dy, dr, r, h, got, dtype, str(wanted))
    assert binding.device_status() == binding.T2S_OK
