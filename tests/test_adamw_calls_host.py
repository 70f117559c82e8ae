"""What the optimizer hands to the library, and what it refuses first, without a GPU."""
import pytest
import torch

from mxfp4_block_scaled_quantize_gb300 import abi, optim

SIZES = (10, 20)


class OnTheGpu(torch.Tensor):
    """Stands for a tensor on GPU 0: its memory is the host's, and nothing reads it there."""
    gpu = 0

    is_cuda = property(lambda self: True)

    def get_device(self):
        return self.gpu


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
