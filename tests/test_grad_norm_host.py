"""What the gradients' norm refuses, and what the optimizer hands to it, without a GPU."""
import ctypes
import math

import pytest
import torch

from mxfp4_block_scaled_quantize_gb300 import abi, optim
from test_adamw_calls_host import SIZES, OnAnotherGpu, tensors


@pytest.fixture(scope="module", autouse=True)
def _lib():
    import __graft_entry__
    __graft_entry__.build()


@pytest.fixture
def calls(monkeypatch):
    """The library's calls, noted instead of made."""
    made = []
    monkeypatch.setattr(abi, "mxfp4_grad_norm", lambda *a, **k: made.append(("norm", a)))
    monkeypatch.setattr(abi, "mxfp4_adamw", lambda *a, **k: made.append(("adamw", a)))
    return made


def test_table_is_the_librarys():
    assert optim._GRADS.itemsize == 16 and optim._GRADS.fields["n"][1] == 8


def call(count=1, g=0x1000, n=8, flags=0, max_norm=1.0, out=0x1000, workspace=0x1000, more=0, table=None):
    lib = abi.load()
    arr = (ctypes.c_uint64 * 4)(g, n, 0x1000, 8)
    need = abi.mxfp4_grad_norm_workspace_bytes(max(0, min(count, abi.MXFP4_GRAD_MAX_TENSORS)))
    address = ctypes.addressof(arr) if table is None else table
    return lib.mxfp4_grad_norm(count, address, flags, max_norm, out, workspace, need + more, None)


@pytest.mark.parametrize("bad", [
    dict(count=-1), dict(count=1, table=0), dict(n=-1 & (2 ** 64 - 1)), dict(n=2 ** 40 + 1), dict(g=0), dict(flags=4), dict(max_norm=0.0),
    dict(max_norm=-1.0), dict(max_norm=math.nan), dict(out=None), dict(workspace=None), dict(more=-1),
    dict(count=2, n=2 ** 40), dict(count=abi.MXFP4_GRAD_MAX_TENSORS + 1)])
def test_arguments_out_of_range_are_refused(bad):
    assert call(**bad) == abi.MXFP4_ERR_INVALID_ARG


@pytest.mark.parametrize("bad", [dict(g=0x1001), dict(g=0x1002, flags=1), dict(out=0x1002), dict(workspace=0x1010)])
def test_misaligned_addresses_are_refused(bad):
    assert call(**bad) == abi.MXFP4_ERR_MISALIGNED


@pytest.mark.parametrize("table, apart", [
    ([(0x1000, 8), (0x1010, 8)], True), ([(0x1010, 8), (0x1000, 8)], True), ([(0x1000, 8), (0x1000, 8)], False),
    ([(0x1000, 9), (0x1010, 8)], False), ([(0x1010, 8), (0x1000, 9)], False), ([(0x2000, 8), (0x1000, 8), (0x1800, 8)], True),
    ([(0x2000, 8), (0x1000, 8), (0x1800, 0x401)], False), ([(0x2000, 8), (0x1000, 0x1000), (0x1800, 4)], False),
    ([(0x1000, 8), (0, 0), (0, 0), (0x1010, 8)], True), ([(0x1000, 8), (0x1004, 0), (0x1010, 8)], True)])
def test_gradients_that_overlap_are_not_scaled(table, apart):
    # the workspace's address is refused after everything else, so that none of the calls launches anything
    arr = (ctypes.c_uint64 * (2 * len(table)))(*[v for pair in table for v in pair])
    need = abi.mxfp4_grad_norm_workspace_bytes(len(table))

    def status(flags):
        return abi.load().mxfp4_grad_norm(len(table), ctypes.addressof(arr), flags, 1.0, 0x1000, 0x1010, need, None)

    assert status(abi.MXFP4_GRAD_SCALE) == (abi.MXFP4_ERR_MISALIGNED if apart else abi.MXFP4_ERR_INVALID_ARG)
    assert status(0) == abi.MXFP4_ERR_MISALIGNED


def test_workspace_grows_with_the_launches():
    sizes = [abi.mxfp4_grad_norm_workspace_bytes(n) for n in (0, 1, 1279, 1280, 2560, abi.MXFP4_GRAD_MAX_TENSORS)]
    assert sizes == sorted(sizes) and sizes[0] > 256 and sizes[2] == sizes[1] and sizes[4] > sizes[3] > sizes[2]
    for bad in (-1, abi.MXFP4_GRAD_MAX_TENSORS + 1):
        with pytest.raises(abi.Mxfp4Error):
            abi.mxfp4_grad_norm_workspace_bytes(bad)


def test_gradients_are_checked(calls):
    norm = optim.GradNorm(tensors())
    for bad in ([], tensors()[:1], tensors(dtype=torch.float16), tensors(torch.Tensor), tensors(OnAnotherGpu),
                [tensors()[0], tensors(dtype=torch.bfloat16)[1]], tensors()[::-1]):
        for f in (norm.measure, norm.clip_):
            with pytest.raises((ValueError, IndexError)):
                f(bad, 1.0)
    for bad in (0.0, -1.0, math.nan):
        with pytest.raises(ValueError):
            norm.clip_(tensors(), bad)
    with pytest.raises(ValueError):
        optim.GradNorm([])
    assert not calls
    assert norm.measure(tensors()) is norm.out
    assert norm.clip_(tensors(dtype=torch.bfloat16), 2.0) is norm.out
    (_, first), (_, second) = calls
    assert first[2:4] == (abi.MXFP4_GRAD_F32, math.inf) and second[2:4] == (abi.MXFP4_GRAD_SCALE, 2.0)


def test_another_current_device_is_refused(calls, monkeypatch):
    norm, opt = optim.GradNorm(tensors()), optim.AdamW(tensors())
    monkeypatch.setattr(abi, "is_current", lambda gpu: gpu != 0)
    for f in (norm.measure, lambda g, m: opt.step(g, max_norm=m)):
        with pytest.raises(ValueError, match="current device"):
            f(tensors(), 1.0)
    assert not calls and opt.steps == 0


def test_a_factor_from_outside_is_checked(calls):
    opt = optim.AdamW(tensors())
    from test_adamw_calls_host import OnTheGpu
    good = torch.ones(1).as_subclass(OnTheGpu)
    for bad in (torch.ones(1), torch.ones(2).as_subclass(OnTheGpu), torch.ones(1, dtype=torch.float64).as_subclass(OnTheGpu),
                torch.ones(1).as_subclass(OnAnotherGpu)):
        with pytest.raises(ValueError, match="grad_factor"):
            opt.step(tensors(), grad_factor=bad)
    with pytest.raises(ValueError, match="grad_factor"):
        opt.step(tensors(), grad_factor=good, max_norm=1.0)
    assert not calls and opt.steps == 0
    opt.step(tensors(), grad_factor=good)
    assert calls[0][1][3].grad_factor == good.data_ptr()


def test_a_step_takes_the_factor_from_the_norm(calls):
    opt = optim.AdamW(tensors())
    grads = tensors()
    opt.step(grads)
    assert [c[0] for c in calls] == ["adamw"] and calls[0][1][3].grad_factor is None
    calls.clear()
    opt.step(grads, max_norm=1.0)
    assert [c[0] for c in calls] == ["norm", "adamw"] and opt.steps == 2
    assert calls[1][1][3].grad_factor == opt.grad_norm.out.data_ptr() + 4
    assert list(opt.grad_norm._table["g"]) == [g.data_ptr() for g in grads] and list(opt.grad_norm._table["n"]) == list(SIZES)
    with pytest.raises(ValueError):
        opt.step(grads, max_norm=0.0)
    assert opt.steps == 2
