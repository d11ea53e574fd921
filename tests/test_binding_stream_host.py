"""The binding's current stream without a GPU: the raw handle where torch has the
private call for it, the public stream object's where it has not."""
import types

import pytest
import torch

from paged_kv_cache_309_gb300 import pa

RAW = "_cuda_getCurrentRawStream"


@pytest.fixture
def device(monkeypatch):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 3)


def test_raw_handle(monkeypatch, device):
    monkeypatch.setattr(torch._C, RAW, lambda d: 0x1000 + d, raising=False)
    assert pa._stream(None) == 0x1003


def test_public_way_back(monkeypatch, device):
    monkeypatch.delattr(torch._C, RAW, raising=False)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda: types.SimpleNamespace(cuda_stream=0x77))
    assert pa._stream(None) == 0x77


def test_a_given_stream(device):
    mine = types.SimpleNamespace(device=torch.device("cuda", 3), cuda_stream=0x55)
    assert pa._stream(mine) == 0x55
    other = types.SimpleNamespace(device=torch.device("cuda", 0), cuda_stream=0x55)
    with pytest.raises(ValueError, match="current device"):
        pa._stream(other)
