"""Streams that the block's calls take (CPU only; stand-ins for tensors and streams of several devices)."""
from types import SimpleNamespace

import pytest
import torch

import moe_grouped_gemm_sizes_amd as mg


def tensor(device):
    return SimpleNamespace(get_device=lambda: device)


def stream(device, handle):
    return SimpleNamespace(device_index=device, cuda_stream=handle)


@pytest.mark.parametrize("current", [0, 1])
def test_stream_of_the_tensors_device(monkeypatch, current):
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: current)
    assert mg._stream_for(tensor(1), stream(1, 77)) == 77
    for handle in (0, 77):                                   # launches would go to the stream's device
        with pytest.raises(ValueError, match="tensors on cuda:1, stream of cuda:0"):
            mg._stream_for(tensor(1), stream(0, handle))


def test_a_default_stream_is_the_current_devices(monkeypatch):
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 1)
    assert mg._stream_for(tensor(1), stream(1, 0)) == 0
    with pytest.raises(ValueError, match="default stream of cuda:0"):
        mg._stream_for(tensor(0), stream(0, 0))
