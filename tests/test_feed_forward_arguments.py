"""Checks of the feed-forward entry points' tensors that need no GPU: CPU tensors stand for a device's."""
from __future__ import annotations

import pytest

torch = pytest.importorskip("torch")

from roofline_driven_tiling_gb300 import binding, feed_forward  # noqa: E402


class OnDevice(torch.Tensor):
    """A CPU tensor that says it lies on GPU `index`."""
    index = 0
    is_cuda = property(lambda self: True)

    def get_device(self):
        return self.index


def on_device(index, shape=(4096,), dtype=torch.uint8):
    t = torch.empty(shape, dtype=dtype).as_subclass(OnDevice)
    t.index = index
    return t


def test_workspace_on_another_device():
    device = torch.device("cuda", 0)
    given = on_device(0)
    assert feed_forward._workspace(given, 0, device, None)[1:] == (given.data_ptr(), 4096)
    with pytest.raises(ValueError, match="workspace"):
        feed_forward._workspace(on_device(1), 0, device, None)
    with pytest.raises(TypeError):
        feed_forward._workspace(torch.empty(4096, dtype=torch.uint8), 0, device, None)
