"""Host-side checks of the AdamW step that need no GPU: its refusals and the table's layout."""
import ctypes

import pytest
import torch

from mxfp4_block_scaled_quantize_gb300 import abi, optim


@pytest.fixture(scope="module")
def lib():
    import __graft_entry__
    __graft_entry__.build()
    return abi.load()


def call(lib, flags=0, count=1, params=None, **change):
    t = dict(p=16, master=None, g=32, m=48, v=64, m_scale=None, v_scale=None, n=10)
    t.update(change)
    arr = (abi.AdamwTensor * 1)(abi.AdamwTensor(*t.values()))
    h = dict(lr=1e-3, beta1=0.9, beta2=0.99, eps=1e-8, weight_decay=0.1, grad_scale=1.0, step=1, dynamic=None)
    h.update(params or {})
    return lib.mxfp4_adamw(count, ctypes.addressof(arr), flags, ctypes.byref(abi.AdamwParams(*h.values())), None)


def test_refusals(lib):
    bad, mis = abi.MXFP4_ERR_INVALID_ARG, abi.MXFP4_ERR_MISALIGNED
    assert call(lib, count=-1) == bad and call(lib, flags=8) == bad
    assert lib.mxfp4_adamw(1, None, 0, None, None) == bad
    for p in ("p", "g", "m", "v"):
        assert call(lib, **{p: None}) == bad
    assert call(lib, n=-1) == bad
    assert call(lib, flags=abi.MXFP4_ADAMW_P_F32, master=80) == bad          # fp32 parameters have no master
    assert call(lib, flags=abi.MXFP4_ADAMW_STATE_E4M3) == bad                # 8-bit moments need scales
    for h in ({"beta1": 1.0}, {"beta2": -0.1}, {"beta1": float("nan")}, {"eps": -1.0}, {"eps": float("inf")},
              {"eps": 1e-40},
              {"step": 0}, {"lr": float("nan")}, {"weight_decay": float("inf")}):
        assert call(lib, params=h) == bad, h
    assert call(lib, p=17) == mis and call(lib, flags=abi.MXFP4_ADAMW_P_F32, p=18) == mis
    assert call(lib, g=33) == mis and call(lib, flags=abi.MXFP4_ADAMW_G_F32, g=34) == mis
    assert call(lib, m=50) == mis and call(lib, master=82) == mis and call(lib, params={"dynamic": 2}) == mis
    assert call(lib, flags=abi.MXFP4_ADAMW_STATE_E4M3, m_scale=80, v_scale=98) == mis


def test_no_usable_device_fails_loudly(lib):
    if torch.cuda.is_available():
        pytest.skip("a CUDA device is present")
    assert call(lib) in (abi.MXFP4_ERR_CUDA, abi.MXFP4_ERR_UNSUPPORTED_DEVICE)


def test_the_table_is_the_c_struct():
    assert optim._TABLE.itemsize == ctypes.sizeof(abi.AdamwTensor)
    for name, _ in abi.AdamwTensor._fields_:
        assert optim._TABLE.fields[name][1] == getattr(abi.AdamwTensor, name).offset


def test_optimizer_refusals():
    p = [torch.zeros(10), torch.zeros(20)]
    with pytest.raises(ValueError):
        optim.AdamW([])
    with pytest.raises(ValueError):
        optim.AdamW([torch.zeros(3, dtype=torch.float16)])
    with pytest.raises(ValueError):
        optim.AdamW(p, masters=p)                          # fp32 parameters
    with pytest.raises(ValueError):
        optim.AdamW(p, state_bits=16)
    with pytest.raises(ValueError):
        optim.AdamW([torch.zeros(4, 5).t()])               # not contiguous
    with pytest.raises(ValueError):
        optim.AdamW(p, exp_avg=[torch.zeros(10)], exp_avg_sq=[torch.zeros(10)])
    opt = optim.AdamW(p)
    for grads in ([torch.zeros(10)], [torch.zeros(10), torch.zeros(21)],
                  [torch.zeros(10), torch.zeros(20, dtype=torch.bfloat16)], [torch.zeros(10), torch.zeros(40)[::2]]):
        with pytest.raises(ValueError):
            opt.step(grads)
    assert opt.steps == 0
