"""Copies of GradNorm and AdamW hand the library tables of their own, without a GPU."""
import copy
import ctypes
import io

import numpy as np
import pytest
import torch

from mxfp4_block_scaled_quantize_gb300 import abi, optim
from test_adamw_calls_host import SIZES, tensors


@pytest.fixture(scope="module", autouse=True)
def _lib():
    import __graft_entry__
    __graft_entry__.build()


@pytest.fixture
def seen(monkeypatch):
    """The tables that the library's calls would read."""
    found = []

    def read(count, address, dtype):
        found.append(np.frombuffer(ctypes.string_at(address, count * dtype.itemsize), dtype=dtype).copy())

    monkeypatch.setattr(abi, "mxfp4_grad_norm", lambda count, address, *a: read(count, address, optim._GRADS))
    monkeypatch.setattr(abi, "mxfp4_adamw", lambda count, address, *a: read(count, address, optim._TABLE))
    return found


def copies(make):
    """Three copies, the original of each gone."""
    yield copy.deepcopy(make())
    file = io.BytesIO()
    torch.save(make(), file)
    file.seek(0)
    yield torch.load(file, weights_only=False)
    yield copy.copy(make())


def plain():
    return [torch.zeros(n) for n in SIZES]


def test_a_copied_norm_reads_its_own_gradients(seen):
    for norm in copies(lambda: optim.GradNorm(plain())):
        norm._gpu = 0   # as if its parameters were there
        others = [np.zeros(len(SIZES), dtype=optim._GRADS) for _ in range(50)]   # what might take an old table's place
        grads = tensors()
        norm.measure(grads)
        table = seen.pop()
        assert list(table["g"]) == [g.data_ptr() for g in grads] and list(table["n"]) == list(SIZES)
        del others


def test_a_copied_optimizer_updates_its_own_tensors(seen):
    for bits in (32, 8):
        for opt in copies(lambda: optim.AdamW([p.bfloat16() for p in plain()], masters=plain(), state_bits=bits, seed=None if bits == 32 else 3)):
            opt._gpu = opt.grad_norm._gpu = 0
            grads = tensors()
            opt.step(grads, max_norm=1.0)
            norm, table = seen
            seen.clear()
            assert list(norm["g"]) == list(table["g"]) == [g.data_ptr() for g in grads]
            assert list(table["p"]) == [p.data_ptr() for p in opt.params] and list(table["master"]) == [p.data_ptr() for p in opt.masters]
            for name, moments in (("m", opt.exp_avg), ("v", opt.exp_avg_sq)):
                codes = moments if bits == 32 else [c for c, _ in moments]
                assert list(table[name]) == [c.data_ptr() for c in codes]
                if bits == 8:
                    assert list(table[name + "_scale"]) == [s.data_ptr() for _, s in moments]
