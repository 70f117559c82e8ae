"""AdamW's parameters from a program that was built before they had a gradient factor, without a GPU."""
import ctypes
import mmap

import pytest

from mxfp4_block_scaled_quantize_gb300 import abi

BEFORE = abi.AdamwParams.grad_factor.offset   # where the structure ended


@pytest.fixture(scope="module", autouse=True)
def _lib():
    import __graft_entry__
    __graft_entry__.build()


def call(flags, behind):
    """The status for parameters with `behind` after the last field that an earlier program knows."""
    h = (ctypes.c_char * ctypes.sizeof(abi.AdamwParams))()
    ctypes.memmove(h, ctypes.byref(abi.AdamwParams(1e-3, 0.9, 0.95, 1e-8, 0.1, 1.0, 1, None, 7)), BEFORE)
    ctypes.memmove(ctypes.addressof(h) + BEFORE, ctypes.byref(ctypes.c_uint64(behind)), 8)
    t = (abi.AdamwTensor * 1)(abi.AdamwTensor(16, None, 32, 48, 64, 80, 96, 0))   # no elements: nothing runs
    return abi.load().mxfp4_adamw(1, ctypes.addressof(t), flags, ctypes.cast(h, ctypes.POINTER(abi.AdamwParams)), None)


@pytest.mark.parametrize("flags", [0, 1, 2, 3, 4, 12, 15])
def test_what_lies_behind_an_earlier_structure_is_not_read(flags):
    plain = call(flags, 0)
    assert plain not in (abi.MXFP4_ERR_INVALID_ARG, abi.MXFP4_ERR_MISALIGNED)
    assert call(flags, 0xDEADBEEF12345677) == plain
    # with the flag it is an address, and checked
    assert call(flags | abi.MXFP4_ADAMW_GRAD_FACTOR, 0) == plain
    assert call(flags | abi.MXFP4_ADAMW_GRAD_FACTOR, 0xDEADBEEF12345677) == abi.MXFP4_ERR_MISALIGNED
    assert call(flags | 64, 0) == abi.MXFP4_ERR_INVALID_ARG


def test_an_earlier_structure_at_the_end_of_its_page():
    # the page behind it cannot be read: a process that tried would end
    page = mmap.PAGESIZE
    both = mmap.mmap(-1, 2 * page)
    at = ctypes.addressof(ctypes.c_char.from_buffer(both))
    libc = ctypes.CDLL(None, use_errno=True)
    assert libc.mprotect(ctypes.c_void_p(at + page), ctypes.c_size_t(page), 0) == 0
    try:
        ctypes.memmove(at + page - BEFORE, ctypes.byref(abi.AdamwParams(1e-3, 0.9, 0.95, 1e-8, 0.1, 1.0, 1, None, 7)), BEFORE)
        h = ctypes.cast(at + page - BEFORE, ctypes.POINTER(abi.AdamwParams))
        t = (abi.AdamwTensor * 1)(abi.AdamwTensor(16, None, 32, 48, 64, 80, 96, 0))
        status = abi.load().mxfp4_adamw(1, ctypes.addressof(t), 0, h, None)
        assert status not in (abi.MXFP4_ERR_INVALID_ARG, abi.MXFP4_ERR_MISALIGNED)
    finally:
        assert libc.mprotect(ctypes.c_void_p(at + page), ctypes.c_size_t(page), mmap.PROT_READ | mmap.PROT_WRITE) == 0


def test_the_optimizer_sets_the_flag(monkeypatch):
    from mxfp4_block_scaled_quantize_gb300 import optim
    from test_adamw_calls_host import OnTheGpu, tensors
    import torch
    made = []
    monkeypatch.setattr(abi, "mxfp4_grad_norm", lambda *a, **k: None)
    monkeypatch.setattr(abi, "mxfp4_adamw", lambda *a, **k: made.append(a))
    opt = optim.AdamW(tensors())
    opt.step(tensors())
    opt.step(tensors(), max_norm=1.0)
    opt.step(tensors(), grad_factor=torch.ones(1).as_subclass(OnTheGpu))
    assert [bool(a[2] & abi.MXFP4_ADAMW_GRAD_FACTOR) for a in made] == [False, True, True]
    assert [a[3].grad_factor is not None for a in made] == [False, True, True]
