"""What layer norm refuses, in the C entries and in the layer, without a GPU."""
import math

import pytest
import torch

from mxfp4_block_scaled_quantize_gb300 import abi
from mxfp4_block_scaled_quantize_gb300.norm import LayerNorm
from test_adamw_calls_host import OnAnotherGpu, OnTheGpu

P = 0x10000


@pytest.fixture(scope="module", autouse=True)
def _lib():
    import __graft_entry__
    __graft_entry__.build()


def forward(x=P, rows=4, dim=64, ldx=64, weight=P, bias=P, samples=1, eps=1e-5, flags=0, y=P, ldy=64, mean=P, rstd=P):
    return abi.load().mxfp4_layer_norm(x, rows, dim, ldx, weight, bias, samples, eps, flags, y, ldy, mean, rstd, None)


def backward(dy=P, lddy=64, x=P, rows=400, dim=64, ldx=64, weight=P, samples=1, flags=0, mean=P, rstd=P, dx=P, lddx=64, dw=P, db=P,
             workspace=P, size=None):
    size = abi.mxfp4_layer_norm_workspace_bytes(64) if size is None else size
    return abi.load().mxfp4_layer_norm_backward(dy, lddy, x, rows, dim, ldx, weight, samples, flags, mean, rstd, dx, lddx, dw, db,
                                                workspace, size, None)


@pytest.mark.parametrize("bad", [
    dict(x=None), dict(y=None), dict(rows=-1), dict(rows=2 ** 40 + 1), dict(dim=0), dict(dim=abi.MXFP4_NORM_MAX_DIM + 1, ldx=2 ** 20, ldy=2 ** 20),
    dict(ldx=63), dict(ldy=63), dict(samples=0), dict(samples=3), dict(eps=-1.0), dict(eps=math.nan), dict(eps=1e39), dict(flags=8),
    dict(mean=None), dict(rstd=None)])
def test_forward_arguments_out_of_range_are_refused(bad):
    assert forward(**bad) == abi.MXFP4_ERR_INVALID_ARG


@pytest.mark.parametrize("bad", [dict(x=P + 1), dict(y=P + 1), dict(x=P + 2, flags=1), dict(weight=P + 1), dict(bias=P + 2, flags=2),
                                 dict(mean=P + 2), dict(rstd=P + 1)])
def test_forward_misaligned_addresses_are_refused(bad):
    assert forward(**bad) == abi.MXFP4_ERR_MISALIGNED


@pytest.mark.parametrize("bad", [
    dict(dy=None), dict(x=None), dict(dx=None), dict(mean=None), dict(rstd=None), dict(rows=-1), dict(dim=0), dict(lddy=63), dict(ldx=63),
    dict(lddx=63), dict(samples=0), dict(samples=3), dict(flags=8), dict(workspace=None), dict(size=100)])
def test_backward_arguments_out_of_range_are_refused(bad):
    assert backward(**bad) == abi.MXFP4_ERR_INVALID_ARG


@pytest.mark.parametrize("bad", [dict(dy=P + 1), dict(x=P + 1), dict(dx=P + 1), dict(weight=P + 2, flags=2), dict(mean=P + 2),
                                 dict(rstd=P + 2), dict(dw=P + 2), dict(db=P + 2), dict(workspace=P + 8)])
def test_backward_misaligned_addresses_are_refused(bad):
    assert backward(**bad) == abi.MXFP4_ERR_MISALIGNED


def test_workspace_refuses_dims_out_of_range():
    for dim in (0, abi.MXFP4_NORM_MAX_DIM + 1):
        with pytest.raises(abi.Mxfp4Error):
            abi.mxfp4_layer_norm_workspace_bytes(dim)


def test_partial_rows_fit_the_workspace():
    # the C entry's sharing out, restated: CTAs with partial rows, over samples and rows, and over the rows from one to the next that
    # starts as far behind a multiple of 16 bytes
    slots = abi.mxfp4_layer_norm_workspace_bytes(1) // 8
    for samples in list(range(1, 320)) + [600, 1000]:
        for each in list(range(1, 40)) + [303, 304, 305, 1000, 4097]:
            rows = samples * each
            chunk = max(-(-rows // 608), 4)
            for period in (1, 2, 4, 8):
                chunks = period * -(-(-(-each // period)) // chunk)
                if period > 1 and samples * chunks > slots:
                    chunks = -(-each // chunk)
                assert chunks == 1 or samples * chunks <= slots


@pytest.fixture
def layer(monkeypatch):
    """A layer on a GPU that is not there, and the library's calls, noted instead of made."""
    made = []
    monkeypatch.setattr(abi, "mxfp4_layer_norm", lambda *a, **k: made.append(a))
    monkeypatch.setattr(abi, "mxfp4_layer_norm_backward", lambda *a, **k: made.append(a))
    one = LayerNorm(64, 12, max_samples=4, device="cpu")
    one._gpu = 0
    one.made = made
    return one


def gpu(*shape, dtype=torch.bfloat16, kind=OnTheGpu):
    return torch.zeros(shape, dtype=dtype).as_subclass(kind)


def test_constructor_refuses():
    for bad in (dict(dim=0), dict(dim=abi.MXFP4_NORM_MAX_DIM + 1), dict(dtype=torch.float16), dict(max_rows=-1), dict(max_samples=0),
                dict(eps=-1.0), dict(eps=math.nan)):
        with pytest.raises(ValueError):
            LayerNorm(**{**dict(dim=64, max_rows=4, device="cpu"), **bad})


@pytest.mark.parametrize("x", [
    gpu(4, 65), gpu(64), gpu(4, 64, dtype=torch.float32), gpu(13, 64), gpu(64, 4).t(), gpu(4, 64, kind=OnAnotherGpu),
    torch.zeros(4, 64, dtype=torch.bfloat16), gpu(64).expand(4, 64)])
def test_rows_are_checked(layer, x):
    with pytest.raises(ValueError):
        layer.forward(x)
    layer.forward(gpu(4, 64))
    layer.made.clear()
    for dy, again in ((x, gpu(4, 64)), (gpu(4, 64), x)):
        with pytest.raises(ValueError):
            layer.backward(dy, again)
    assert not layer.made


@pytest.mark.parametrize("v", [
    gpu(63), gpu(4, 63), gpu(3, 64), gpu(6, 64), gpu(0, 64), gpu(1, 1, 64), gpu(64, dtype=torch.float16), gpu(128)[::2],
    gpu(64, kind=OnAnotherGpu), torch.zeros(64)])
def test_vectors_are_checked(layer, v):
    for args in ((v, None), (None, v)):
        with pytest.raises(ValueError):
            layer.forward(gpu(4, 64), *args)
    assert not layer.made


def test_vectors_of_two_kinds_are_refused(layer):
    for w, b in ((gpu(64), gpu(64, dtype=torch.float32)), (gpu(2, 64), gpu(64)), (gpu(2, 64), gpu(4, 64))):
        with pytest.raises(ValueError):
            layer.forward(gpu(4, 64), w, b)
    assert not layer.made


def test_another_current_device_is_refused(layer, monkeypatch):
    layer.forward(gpu(4, 64))
    layer.made.clear()
    monkeypatch.setattr(abi, "is_current", lambda gpu: gpu != 0)
    for f in (lambda: layer.forward(gpu(4, 64)), lambda: layer.backward(gpu(4, 64), gpu(4, 64))):
        with pytest.raises(ValueError, match="current device"):
            f()
    assert not layer.made


def test_backward_goes_with_the_last_forward(layer):
    x, w = gpu(4, 64), gpu(2, 64)
    with pytest.raises(ValueError, match="no forward"):
        layer.backward(x, x)
    layer.forward(x, w)
    for args in ((x, x), (gpu(3, 64), x, w), (x, gpu(3, 64), w), (x, x, gpu(64)), (x, x, gpu(2, 64, dtype=torch.float32))):
        with pytest.raises(ValueError):
            layer.backward(*args)
    dx, dw, db = layer.backward(x, x, w)
    assert dx.shape == (4, 64) and dw.shape == (2, 64) and db is None
    layer.forward(x, None, gpu(64))
    dx, dw, db = layer.backward(x, x)
    assert dw is None and db.shape == (64,)
    layer.train = False
    with pytest.raises(ValueError, match="training"):
        layer.backward(x, x)
