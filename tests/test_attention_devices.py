"""The attention binding's check of devices, without a GPU: the library
launches on the current device, so tensors and streams of another are refused
before it is called."""
import pytest
import torch

from nvfp4_block_scaled_gather_gb300 import attention as A


class Stream:
    def __init__(self, index, handle=77):
        self.device, self.cuda_stream = torch.device("cuda", index), handle


@pytest.fixture
def current(monkeypatch):
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 1)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda device: 1000 + device)


def test_the_current_device_is_the_tensors(current):
    assert A._stream(None, 1) == 1001 and A._stream(Stream(1), 1) == 77
    with pytest.raises(ValueError, match="current device is cuda:1"):
        A._stream(None, 0)
    with pytest.raises(ValueError, match="current device is cuda:1"):
        A._stream(Stream(0), 0)


def test_the_stream_is_on_the_tensors_device(current):
    with pytest.raises(ValueError, match="stream's device is cuda:0"):
        A._stream(Stream(0), 1)
