"""What the few tokens' layer of experts refuses, in the C entry and in the layer, without a GPU."""
import pytest
import torch

from mxfp4_block_scaled_quantize_gb300 import abi
from mxfp4_block_scaled_quantize_gb300.experts import MXFP4Experts
from test_adamw_calls_host import OnAnotherGpu, OnTheGpu

P = 0x10000
SIZES = dict(tokens=4, experts=8, top_k=2, dim=256, inner=128)


@pytest.fixture(scope="module", autouse=True)
def _lib():
    import __graft_entry__
    __graft_entry__.build()


def call(x=P, tokens=4, ldx=256, logits=P, ldl=8, experts=8, top_k=2, dim=256, inner=128, up_q=P, up_s=P, down_q=P, down_s=P, y=P,
         ldy=256, flags=0, workspace=P, size=None):
    size = abi.mxfp4_experts_workspace_bytes(**SIZES) if size is None else size
    return abi.load().mxfp4_experts_forward(x, tokens, ldx, logits, ldl, experts, top_k, dim, inner, up_q, up_s, down_q, down_s, y, ldy,
                                            flags, workspace, size, None)


@pytest.mark.parametrize("bad", [
    dict(x=None), dict(logits=None), dict(up_q=None), dict(up_s=None), dict(down_q=None), dict(down_s=None), dict(y=None),
    dict(workspace=None), dict(size=1000), dict(tokens=-1), dict(tokens=abi.MXFP4_EXPERTS_MAX_TOKENS + 1), dict(experts=0),
    dict(experts=abi.MXFP4_MAX_GROUPS + 1, ldl=2000), dict(top_k=0), dict(top_k=9), dict(experts=40, ldl=40, top_k=17), dict(dim=0), dict(inner=0),
    dict(dim=70000, ldx=70000, ldy=70000), dict(inner=70000), dict(ldx=255), dict(ldy=255), dict(ldl=7), dict(flags=4), dict(ldx=2 ** 41)])
def test_arguments_out_of_range_are_refused(bad):
    assert call(**bad) == abi.MXFP4_ERR_INVALID_ARG


@pytest.mark.parametrize("bad", [
    dict(x=P + 1), dict(y=P + 1), dict(logits=P + 1), dict(logits=P + 2, flags=1), dict(up_q=P + 8), dict(up_s=P + 4), dict(down_q=P + 8),
    dict(down_s=P + 8), dict(workspace=P + 128)])
def test_misaligned_addresses_are_refused(bad):
    assert call(**bad) == abi.MXFP4_ERR_MISALIGNED


def test_workspace_tells_what_fits():
    for t in (0, 1, 8, 9, 64):
        for experts, top_k in ((1, 1), (64, 8), (1024, 16)):
            assert abi.mxfp4_experts_workspace_bytes(t, experts, top_k, 7040, 3456) >= 4 * t * top_k * 10496
    for bad in (dict(dim=12000), dict(inner=6000), dict(tokens=65), dict(top_k=9), dict(experts=0)):
        with pytest.raises(abi.Mxfp4Error):
            abi.mxfp4_experts_workspace_bytes(**{**SIZES, **bad})


def test_constructor_refuses():
    for bad in (dict(top_k=0), dict(top_k=9), dict(experts=40, top_k=17), dict(max_tokens=0), dict(max_tokens=65)):
        with pytest.raises(ValueError):
            MXFP4Experts(**{**dict(experts=8, dim=256, inner=128, top_k=2, device="cpu"), **bad})
    for bad in (dict(dim=0), dict(inner=0), dict(dim=12000), dict(inner=6000), dict(experts=2000)):
        with pytest.raises(abi.Mxfp4Error):
            MXFP4Experts(**{**dict(experts=8, dim=256, inner=128, top_k=2, device="cpu"), **bad})


def gpu(*shape, dtype=torch.bfloat16, kind=OnTheGpu):
    return torch.zeros(shape, dtype=dtype).as_subclass(kind)


@pytest.fixture
def layer(monkeypatch):
    """A layer on a GPU that is not there, and the library's calls, noted instead of made."""
    made = []
    monkeypatch.setattr(abi, "mxfp4_experts_forward", lambda *a, **k: made.append(a))
    one = MXFP4Experts(8, 256, 128, 2, max_tokens=6, device="cpu")
    one._gpu = 0
    one.made = made
    one.blobs = [gpu(n, dtype=torch.uint8) for n in one._bytes]
    return one


@pytest.mark.parametrize("x", [gpu(4, 255), gpu(256), gpu(7, 256), gpu(4, 256, dtype=torch.float32), gpu(256, 4).t(), gpu(256).expand(4, 256),
                               gpu(4, 256, kind=OnAnotherGpu), torch.zeros(4, 256, dtype=torch.bfloat16), gpu(3, 256)])
def test_x_is_checked(layer, x):
    with pytest.raises(ValueError):
        layer.forward(x, gpu(4 if x.shape[0] != 7 else 7, 8), *layer.blobs)
    assert not layer.made


@pytest.mark.parametrize("logits", [gpu(4, 7), gpu(8), gpu(5, 8), gpu(4, 8, dtype=torch.float16), gpu(8, 4).t(),
                                    gpu(4, 8, kind=OnAnotherGpu), torch.zeros(4, 8), gpu(8).expand(4, 8)])
def test_logits_are_checked(layer, logits):
    with pytest.raises(ValueError):
        layer.forward(gpu(4, 256), logits, *layer.blobs)
    assert not layer.made


def test_another_current_device_is_refused(layer, monkeypatch):
    monkeypatch.setattr(abi, "is_current", lambda gpu: gpu != 0)
    with pytest.raises(ValueError, match="current device"):
        layer.forward(gpu(4, 256), gpu(4, 8), *layer.blobs)
    assert not layer.made


@pytest.mark.parametrize("which", range(4))
def test_packed_weights_are_checked(layer, which):
    n = layer._bytes[which]
    for bad in (gpu(n - 1, dtype=torch.uint8), gpu(n), gpu(2 * n, dtype=torch.uint8)[::2], gpu(n, dtype=torch.uint8, kind=OnAnotherGpu), None,
                torch.zeros(n, dtype=torch.uint8)):
        blobs = list(layer.blobs)
        blobs[which] = bad
        with pytest.raises(ValueError):
            layer.forward(gpu(4, 256), gpu(4, 8), *blobs)
    assert not layer.made
    assert layer.forward(gpu(4, 256), gpu(4, 8), *layer.blobs).shape == (4, 256)
    assert layer.forward(gpu(6, 256), gpu(6, 8, dtype=torch.float32), *layer.blobs).shape == (6, 256)
    assert [c[15] for c in layer.made] == [abi.MXFP4_EXPERTS_NORMALIZE, abi.MXFP4_EXPERTS_NORMALIZE | abi.MXFP4_EXPERTS_LOGITS_F32]
