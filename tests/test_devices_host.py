"""Calls on another device than the current one: refused before the library sees an address (fake tensors and streams,
no GPU)."""

import pytest
import torch

from segmented_gather_gemm_lora_gb300 import binding as B


class On:
    """Stands for a tensor on a CUDA device."""

    def __init__(self, device):
        self.device = device

    def get_device(self):
        return self.device


class Stream:
    """Stands for a stream of a device."""

    def __init__(self, device):
        self.device_index, self.cuda_stream = device, 100 + device


@pytest.fixture
def two_devices(monkeypatch):
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda d: 10 + d, raising=False)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch.cuda, "Stream", Stream)


def test_calls_on_the_current_device(two_devices):
    assert B._one_device(None, On(0), None, On(0)) == 10
    assert B._one_device(Stream(0), On(0), On(0)) == 100
    assert B._one_device(7, On(0)) == 7


@pytest.mark.parametrize("stream", [None, 7, Stream(0), Stream(1)])
def test_tensors_of_another_device_than_the_current_one(two_devices, stream):
    with pytest.raises(ValueError):
        B._one_device(stream, On(1), On(1))


def test_a_stream_of_another_device_than_the_tensors(two_devices):
    with pytest.raises(ValueError):
        B._one_device(Stream(1), On(0), On(0))


@pytest.mark.parametrize("stream", [None, 7, Stream(0)])
def test_tensors_of_two_devices_or_none(two_devices, stream):
    with pytest.raises(ValueError):
        B._one_device(stream, On(0), On(1))
    with pytest.raises(ValueError):
        B._one_device(stream, On(-1), On(-1))
