"""The handle of the current stream, whatever names this torch has for it."""
import pytest
import torch

from mxfp4_block_scaled_quantize_gb300 import abi

NAMES = ("_cuda_getCurrentRawStream", "_cuda_getDevice")


@pytest.mark.parametrize("missing", [(), NAMES[:1], NAMES[1:], NAMES])
def test_current_stream(monkeypatch, missing):
    class Stream:
        cuda_stream = 77

    monkeypatch.setattr(abi, "_current_stream", None, raising=False)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda: Stream)
    monkeypatch.setattr(torch._C, NAMES[0], lambda device: 70 + device, raising=False)
    monkeypatch.setattr(torch._C, NAMES[1], lambda: 7, raising=False)
    for name in missing:
        monkeypatch.delattr(torch._C, name)
    for _ in range(2):
        assert abi._stream(None) == 77
    assert abi._stream(5) == 5 and abi._stream(Stream) == 77


@pytest.mark.gpu
def test_current_stream_is_the_public_one(monkeypatch):
    monkeypatch.setattr(abi, "_current_stream", None)
    side = torch.cuda.Stream()
    assert abi._stream(None) == torch.cuda.current_stream().cuda_stream
    with torch.cuda.stream(side):
        assert abi._stream(None) == side.cuda_stream == torch.cuda.current_stream().cuda_stream
