"""Which stream a call without one takes (no GPU: torch's side is stood in for)."""
import types

import pytest
import torch

import collective_window_put_amd as vr


@pytest.fixture
def fake(monkeypatch):
    monkeypatch.setattr(torch.cuda, "is_initialized", lambda: True)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 3)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda: types.SimpleNamespace(cuda_stream=0x50))
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 3, raising=False)
    return monkeypatch


def test_the_current_stream_of_the_current_device(fake):
    fake.setattr(torch._C, "_cuda_getCurrentRawStream", lambda device: 0x40 + device, raising=False)
    assert vr._stream(None) == 0x43
    fake.setattr(torch.cuda, "is_initialized", lambda: False)
    assert vr._stream(None) == 0x50


def test_a_torch_without_the_raw_call(fake):
    # the raw call is not part of torch's public interface
    fake.delattr(torch._C, "_cuda_getCurrentRawStream", raising=False)
    fake.delattr(torch._C, "_cuda_getDevice", raising=False)
    assert vr._stream(None) == 0x50


def test_given_streams():
    assert vr._stream(0x70) == 0x70
    assert vr._stream(types.SimpleNamespace(cuda_stream=0x60)) == 0x60
