"""GPU: the gradients' norm, clipping and the clipped AdamW step over lists with empty tensors where one launch's table ends.

The tolerances are those of the norm's own tests: u = 2^-24, 17 u for norm and factor, half a step of the type and 18 u for a clipped
gradient."""
import math

import numpy as np
import pytest
import torch

from mxfp4_block_scaled_quantize_gb300 import abi
from mxfp4_block_scaled_quantize_gb300.optim import AdamW, GradNorm

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
LISTS = [[5] * 1280 + [0], [5] * 1280 + [0] * 7, [0] * 2 + [3] * 1280 + [0], [5] * 2560 + [0], [5] * 1280 + [0] * 3 + [7]]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    import __graft_entry__
    __graft_entry__.build()
    torch.cuda.set_device(0)
    yield
    assert abi.mxfp4_last_device_error() == abi.MXFP4_OK


def gradients(sizes, dtype):
    flat = torch.randn(sum(sizes), generator=torch.Generator(device="cuda").manual_seed(len(sizes)), device="cuda").to(TYPES[dtype])
    return flat, list(flat.split(sizes))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("sizes", LISTS, ids=lambda s: f"{len(s)}_of_which_{sum(n > 0 for n in s)}")
def test_norm_and_clipping(dtype, sizes):
    flat, grads = gradients(sizes, dtype)
    before = flat.cpu().double().numpy()
    norm = math.sqrt(float(before @ before))
    factor = 1.0 / (norm + 1e-6)
    g = GradNorm(grads)
    for run in (g.measure, g.measure, g.clip_):   # a call finds the workspace as the one before left it
        out = run(grads, 1.0).tolist()
        assert abs(out[0] - norm) <= 17 * U * norm and abs(out[1] - factor) <= 17 * U * factor
    half = U if dtype == "f32" else 2.0 ** -8
    assert np.all(np.abs(flat.cpu().double().numpy() - before * factor) <= (half + 18 * U) * np.abs(before * factor))


@pytest.mark.parametrize("sizes", LISTS[:2], ids=len)
def test_clipped_step(sizes):
    flat, grads = gradients(sizes, "f32")
    params = [torch.ones(n, device="cuda") for n in sizes]
    clipped, plain = AdamW([p.clone() for p in params], lr=1e-2), AdamW(params, lr=1e-2)
    clipped.step(grads, max_norm=0.5)
    plain.step(grads, grad_scale=clipped.grad_norm.out[1].item())
    norm = float(flat.double().norm())
    assert abs(clipped.grad_norm.out[0].item() - norm) <= 17 * U * norm
    assert all(torch.equal(a, b) for a, b in zip(clipped.params, plain.params))
