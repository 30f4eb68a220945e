"""Tensors on another device than the current one, on which the kernels run, are
refused: their addresses may not be valid there.  With stand-ins for tensors of a
second device, so this runs without a GPU."""
import pytest
import torch

from combine_ep_get_04_gb300 import _tensors


class Tensor:
    dtype, shape, is_cuda = torch.float32, torch.Size((4, 8)), True

    def __init__(self, device):
        self.at = device
        self.device = torch.device("cuda", device)

    def get_device(self):
        return self.at

    def stride(self):
        return 8, 1

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return 0x1000


CALLS = {"rows": lambda t: _tensors._rows_ptr(t, torch.float32, "x", (4, 8)), "shaped": lambda t: _tensors._shaped_ptr(t, torch.float32, "x", (4, 8))}


@pytest.mark.parametrize("which", CALLS)
def test_tensors_of_another_device(which, monkeypatch):
    monkeypatch.setattr(_tensors, "_SEVERAL", True, raising=False)
    monkeypatch.setattr(_tensors, "_current_device", lambda: 0)
    call = CALLS[which]
    assert call(Tensor(0)) in ((0x1000, 8), 0x1000)
    with pytest.raises(ValueError, match="x is on cuda:1, the current device is cuda:0"):
        call(Tensor(1))
    monkeypatch.setattr(_tensors, "_current_device", lambda: 1)
    assert call(Tensor(1)) in ((0x1000, 8), 0x1000)


def test_what_an_object_holds(monkeypatch):
    """The buffers of a LayerNorm and packed weights, which are made before the call."""
    monkeypatch.setattr(_tensors, "_SEVERAL", True, raising=False)
    monkeypatch.setattr(_tensors, "_current_device", lambda: 0)
    _tensors._on_current(Tensor(0), "the norm")
    with pytest.raises(ValueError, match="the norm is on cuda:1, the current device is cuda:0"):
        _tensors._on_current(Tensor(1), "the norm")
    monkeypatch.setattr(_tensors, "_SEVERAL", False)
    _tensors._on_current(Tensor(1), "the norm")           # one device: nothing to look at
