"""GPU: norm and factor of gradients that are not finite, for a finite and for an infinite largest norm."""
import math

import pytest
import torch

from mxfp4_block_scaled_quantize_gb300 import abi
from mxfp4_block_scaled_quantize_gb300.optim import AdamW, GradNorm

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    import __graft_entry__
    __graft_entry__.build()
    torch.cuda.set_device(0)
    yield
    assert abi.mxfp4_last_device_error() == abi.MXFP4_OK


def gradients(dtype, bad):
    grads = [torch.full((n,), 0.25, dtype=dtype, device="cuda") for n in (9000, 7, 300)]
    grads[1][6] = bad
    return grads


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_a_nan_makes_both_nan(dtype):
    for args in ((), (math.inf,), (1.0,), (1e30,)):
        out = GradNorm(gradients(dtype, 0.0)).measure(gradients(dtype, math.nan), *args)
        assert torch.isnan(out).all()
    for max_norm in (math.inf, 2.0):
        grads = gradients(dtype, math.nan)
        assert torch.isnan(GradNorm(grads).clip_(grads, max_norm)).all()
        assert all(torch.isnan(g).all() for g in grads)   # times a factor of NaN


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("bad", [math.inf, -math.inf])
def test_an_infinity(dtype, bad):
    grads = gradients(dtype, bad)
    norm = GradNorm(grads)
    assert norm.measure(grads).tolist() == [math.inf, 1.0]   # no largest norm: nothing to scale down to
    assert norm.measure(grads, math.inf).tolist() == [math.inf, 1.0]
    assert norm.measure(grads, 2.0).tolist() == [math.inf, 0.0]
    kept = [g.clone() for g in grads]
    norm.clip_(grads, math.inf)
    assert all(torch.equal(g, k) for g, k in zip(grads, kept))


def test_a_step_takes_the_nan():
    params = [torch.ones(n, device="cuda") for n in (9000, 7, 300)]
    opt = AdamW(params, lr=1e-2)
    opt.step(gradients(torch.float32, math.nan), max_norm=math.inf)
    assert torch.isnan(opt.grad_norm.out).all() and all(torch.isnan(p).all() for p in params)
