"""What the optimizer hands to the library, and what it refuses first, without a GPU."""
import ctypes

import pytest
import torch

from mxfp4_block_scaled_quantize_gb300 import abi, optim

SIZES = (10, 20)


@pytest.fixture(scope="module", autouse=True)
def _lib():
    import __graft_entry__
    __graft_entry__.build()


class OnTheGpu(torch.Tensor):
    """Stands for a tensor on GPU 0: its memory is the host's, and nothing reads it there."""
    gpu = 0

    is_cuda = property(lambda self: True)

    def get_device(self):
        return self.gpu

    @classmethod
    def __torch_function__(cls, func, types, args=(), kwargs=None):
        if func is torch.Tensor.get_device:   # called as a function
            return args[0].gpu
        return super().__torch_function__(func, types, args, kwargs or {})


class OnAnotherGpu(OnTheGpu):
    gpu = 1


def tensors(kind=OnTheGpu, dtype=torch.float32):
    return [torch.zeros(n, dtype=dtype).as_subclass(kind) for n in SIZES]


@pytest.fixture
def calls(monkeypatch):
    """The library's calls, noted instead of made."""
    made = []
    monkeypatch.setattr(abi, "mxfp4_adamw", lambda *a, **k: made.append(a))
    return made


def test_gradients_elsewhere_are_refused(calls):
    # a host address would be dereferenced on the GPU
    opt = optim.AdamW(tensors())
    for bad in (torch.Tensor, OnAnotherGpu):
        for j in (0, 1):
            grads = tensors()
            grads[j] = torch.zeros(SIZES[j]).as_subclass(bad)
            with pytest.raises(ValueError, match="GPU"):
                opt.step(grads)
    assert not calls and opt.steps == 0
    opt.step(tensors())
    assert len(calls) == 1 and opt.steps == 1


def test_parameters_on_the_host_are_refused(calls):
    opt = optim.AdamW([torch.zeros(10)])
    with pytest.raises(ValueError, match="GPU"):
        opt.step([torch.zeros(10)])
    assert not calls and opt.steps == 0


def test_values_on_the_device_are_four_in_a_row(calls):
    opt = optim.AdamW(tensors())
    four = torch.zeros(4).as_subclass(OnTheGpu)
    for bad in (torch.zeros(8).as_subclass(OnTheGpu)[::2], torch.zeros(4), four.double(), torch.zeros(5).as_subclass(OnTheGpu),
                torch.zeros(4).as_subclass(OnAnotherGpu)):
        with pytest.raises(ValueError, match="dynamic"):
            opt.step(tensors(), dynamic=bad)
    assert not calls and opt.steps == 0
    opt.step(tensors(), dynamic=four)
    assert calls[0][3].dynamic == four.data_ptr()


def test_a_refused_step_does_not_count(calls, monkeypatch):
    opt = optim.AdamW(tensors())
    opt.step(tensors())

    def refuse(*args):
        raise abi.Mxfp4Error(abi.MXFP4_ERR_INVALID_ARG, "mxfp4_adamw")

    with monkeypatch.context() as m:
        m.setattr(abi, "mxfp4_adamw", refuse)
        for step in (None, 7):
            with pytest.raises(abi.Mxfp4Error):
                opt.step(tensors(), step=step, lr=float("nan"))
            assert opt.steps == 1
    opt.step(tensors())
    assert opt.steps == 2 and calls[-1][3].step == 2
    opt.step(tensors(), step=7)
    assert opt.steps == 7 and calls[-1][3].step == 7


def test_moments_come_both_or_not_at_all():
    p = tensors()
    m32 = tensors()
    m8 = [(torch.zeros(n, dtype=torch.float8_e4m3fn).as_subclass(OnTheGpu), torch.zeros(1).as_subclass(OnTheGpu))
          for n in SIZES]
    for m, v in ((m32, None), (None, m32), (m8, None), (m32, m8), (m8, m32), ([m32[0], m8[1]], m32), (m8, [m8[0], m32[1]]),
                 (m8, [m8[0], m8[1] + m8[1]])):
        with pytest.raises(ValueError):
            optim.AdamW(p, exp_avg=m, exp_avg_sq=v)
    assert optim.AdamW(p, exp_avg=m32, exp_avg_sq=m32).state_bits == 32
    assert optim.AdamW(p, exp_avg=m8, exp_avg_sq=m8).state_bits == 8


def moments8():
    return [(torch.zeros(n, dtype=torch.float8_e4m3fn).as_subclass(OnTheGpu), torch.zeros(1).as_subclass(OnTheGpu))
            for n in SIZES]


def test_codes_to_nearest_are_for_a_fast_second_moment(calls):
    # at beta2 = 0.999 a code never moves by itself
    kinds = ({"state_bits": 8}, {"exp_avg": moments8(), "exp_avg_sq": moments8()})
    for kind in kinds:
        with pytest.raises(ValueError, match="seed"):
            optim.AdamW(tensors(), betas=(0.9, 0.999), **kind)
        assert optim.AdamW(tensors(), **kind).betas == (0.9, 0.95)
        assert optim.AdamW(tensors(), betas=(0.8, 0.95), **kind).betas == (0.8, 0.95)
        assert optim.AdamW(tensors(), seed=3, **kind).betas == (0.9, 0.999)
        opt = optim.AdamW(tensors(), betas=(0.9, 0.9999), seed=-1, **kind)
        opt.step(tensors())
        _, _, flags, h, _ = calls[-1]
        assert flags & abi.MXFP4_ADAMW_STOCHASTIC and h.seed == 2 ** 64 - 1
    assert optim.AdamW(tensors()).betas == (0.9, 0.999)
    with pytest.raises(ValueError, match="8-bit"):
        optim.AdamW(tensors(), seed=0)


def test_stochastic_rounding_wants_the_step_among_the_values_on_the_device(calls):
    opt = optim.AdamW(tensors(), state_bits=8, seed=0)
    with pytest.raises(ValueError, match="5 consecutive"):
        opt.step(tensors(), dynamic=torch.zeros(4).as_subclass(OnTheGpu))
    opt.step(tensors(), dynamic=torch.zeros(5).as_subclass(OnTheGpu))


def test_the_library_refuses_what_it_cannot_follow():
    lib = abi.load()
    e4m3, sr = abi.MXFP4_ADAMW_STATE_E4M3, abi.MXFP4_ADAMW_STOCHASTIC
    t = (abi.AdamwTensor * 1)(abi.AdamwTensor(16, None, 32, 48, 64, 80, 96, 0))   # no elements: nothing would run

    def call(flags, beta2):
        h = abi.AdamwParams(1e-3, 0.9, beta2, 1e-8, 0.1, 1.0, 1, None, 7)
        return lib.mxfp4_adamw(1, ctypes.addressof(t), flags, ctypes.byref(h), None)

    bad = abi.MXFP4_ERR_INVALID_ARG
    for beta2 in (0.951, 0.99, 0.999):
        assert call(e4m3, beta2) == bad
        assert call(e4m3 | sr, beta2) != bad and call(0, beta2) != bad
    assert call(e4m3, 0.95) != bad
    for flags in (sr, sr | 1, sr | 3, 16, 16 | e4m3):   # stochastic rounding is of 8-bit moments
        assert call(flags, 0.9) == bad
