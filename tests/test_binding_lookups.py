"""The binding's lookups of the current device and stream, with torch's quick (private) ones and without them."""
import types

import pytest
import torch

from lossless_entropy_coded_amd import wc


@pytest.fixture()
def device(monkeypatch):
    """torch as with device 3 in use and stream 77 current on it."""
    for name, value in list(vars(wc).items()):
        if name in ("_torch", "_lookups_found"):
            monkeypatch.setattr(wc, name, None)       # (what earlier calls found)
    monkeypatch.setattr(torch.cuda, "is_initialized", lambda: True)
    monkeypatch.setattr(torch.cuda, "is_available", lambda: True)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 3)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: types.SimpleNamespace(cuda_stream=77))
    return monkeypatch


def test_without_the_private_names(device):
    device.delattr(torch._C, "_cuda_getDevice", raising=False)
    device.delattr(torch._C, "_cuda_getCurrentRawStream", raising=False)
    for _ in range(2):
        assert wc._current_device() == 3
        assert wc._stream_handle(None) == 77
    assert wc._stream_handle(5) == 5
    assert wc._stream_handle(types.SimpleNamespace(cuda_stream=9)) == 9


def test_with_the_private_names(device):
    device.setattr(torch._C, "_cuda_getDevice", lambda: 3, raising=False)
    device.setattr(torch._C, "_cuda_getCurrentRawStream", lambda d: 70 + d, raising=False)
    assert wc._current_device() == 3
    assert wc._stream_handle(None) == 73


def test_before_a_device_is_in_use(device):
    """Nothing is kept from a lookup before torch has a device in use."""
    device.setattr(torch.cuda, "is_initialized", lambda: False)
    assert wc._current_device() == 3 and wc._stream_handle(None) == 77
    device.setattr(torch.cuda, "is_available", lambda: False)
    assert wc._current_device() is None
