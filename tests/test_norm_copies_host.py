"""Copies of a LayerNorm return views of their own buffers, without a GPU."""
import copy
import pickle

import pytest

from mxfp4_block_scaled_quantize_gb300 import abi
from mxfp4_block_scaled_quantize_gb300.norm import LayerNorm
from test_norm_host import gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    import __graft_entry__
    __graft_entry__.build()


def test_a_copied_layer_returns_views_of_its_own_buffers(monkeypatch):
    made = []
    monkeypatch.setattr(abi, "mxfp4_layer_norm", lambda *a, **k: made.append(a))
    monkeypatch.setattr(abi, "mxfp4_layer_norm_backward", lambda *a, **k: made.append(a))
    layer = LayerNorm(64, 12, device="cpu")
    layer._gpu = 0
    x, w = gpu(4, 64), gpu(64)
    layer.forward(x, w, w)
    first = layer.backward(x, x, w)
    for other in (copy.deepcopy(layer), pickle.loads(pickle.dumps(layer))):
        dx, dw, db = other.backward(x, x, w)
        assert dx.data_ptr() == other.dx.data_ptr() != layer.dx.data_ptr()
        assert dw.data_ptr() == other.dw.data_ptr() and db.data_ptr() == other.db.data_ptr()
        assert made[-1][13] is other.dw and made[-1][14] is other.db
    again = copy.copy(layer).backward(x, x, w)   # shares the buffers
    assert [t.data_ptr() for t in again] == [t.data_ptr() for t in first]
    serving = copy.deepcopy(LayerNorm(64, 12, train=False, device="cpu"))
    assert serving.mean is None and not serving.train
