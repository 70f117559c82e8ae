"""GPU: the few tokens' experts at the ends of what they state of their numbers: scales up to 2^96, and x in fp16 under one power of two.

Tolerances, derived before the first run: one product of n equal terms is off by 160 u of its value (u = 2^-24; additions of a block's
matrix instructions, its scale, and the blocks after one another), silu(g) u by 1.1 and 1 times that and 12 u, h by 2^-22 more; together
below 600 u + 2^-22 < 4e-5 of the value, where all terms have one sign; and y by half a step of bf16, 2^-8."""
import numpy as np
import pytest
import torch

from mxfp4_block_scaled_quantize_gb300 import abi
from mxfp4_block_scaled_quantize_gb300.experts import MXFP4Experts
from test_gpu_few_experts import Problem

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    import __graft_entry__
    __graft_entry__.build()
    torch.cuda.set_device(0)
    yield
    assert abi.mxfp4_last_device_error() == abi.MXFP4_OK


def blob(rows, k, code, byte):
    """One expert's weights, all `code` times 2^(byte - 127)."""
    kp, rows_up = -(-k // 128) * 128, -(-rows // 128) * 128
    q = torch.zeros(rows, kp // 2, dtype=torch.uint8, device="cuda")
    q[:, :k // 2] = code | code << 4
    return q, torch.full((rows_up * kp // 32,), byte, dtype=torch.uint8, device="cuda")


@pytest.mark.parametrize("tokens", [1, 4, 12])
@pytest.mark.parametrize("dim, inner", [(7040, 64), (256, 3456)])
@pytest.mark.parametrize("which", ["up", "down"])
def test_the_largest_sums_of_the_largest_scales(tokens, dim, inner, which):
    # codes of 6 and a row of x of one value just below a power of two: no sum of that many elements is larger
    x_value, up_byte, down_byte = ((2 - 2 ** -7) * 2.0 ** -101, 223, 127) if which == "up" else ((2 - 2 ** -7) * 2.0 ** -60, 127, 223)
    layer = MXFP4Experts(1, dim, inner, 1, max_tokens=tokens)
    x = torch.full((tokens, dim), x_value, dtype=torch.bfloat16, device="cuda")
    y = layer.forward(x, torch.zeros(tokens, 1, device="cuda"), *blob(2 * inner, dim, 7, up_byte), *blob(dim, inner, 7, down_byte))
    g = 6 * 2.0 ** (up_byte - 127) * dim * x_value
    h = g / (1 + np.exp(-g)) * g
    want = 6 * 2.0 ** (down_byte - 127) * inner * h
    assert 2.0 ** -126 < want < 3e38
    got = y.double()
    assert ((got - want).abs() <= (4e-5 + 2.0 ** -8) * want).all()


@pytest.mark.parametrize("tokens", [2, 12])
@pytest.mark.parametrize("x_scale, std", [(2.0 ** -110, 2.0 ** 90), (2.0 ** -125, 2.0 ** 92), (2.0 ** 60, 2.0 ** -40)])
def test_random_values_near_the_ends(x_scale, std, tokens):
    p = Problem(tokens, 4, 2, 256, 128, seed=31, x_scale=x_scale, std=std)
    p.check(p.run(p.layer()))


@pytest.mark.parametrize("tokens", [3, 12])
@pytest.mark.parametrize("down", [28, 31, 35, 39, 45])
def test_small_elements_of_a_row_with_a_large_one(tokens, down):
    # weights that see the small elements alone: what is exact from 2^-31 of the largest on, and off by 2^-39 of it below
    dim, inner = 256, 32
    g = torch.Generator(device="cuda").manual_seed(down)
    x = (2.0 ** -down * (1 + torch.rand(tokens, dim, generator=g, device="cuda"))).to(torch.bfloat16)
    x[:, :32] = 1.0
    up = blob(2 * inner, dim, 2, 127)   # ones
    up[0][:, :16] = 0                   # and zeros for the first 32
    layer = MXFP4Experts(1, dim, inner, 1, max_tokens=tokens)
    # W1's rows of u as W2's, so that y_r = inner silu(g) u 2^60
    y = layer.forward(x, torch.zeros(tokens, 1, device="cuda"), *up, *blob(dim, inner, 2, 187)).double()
    s = x[:, 32:].double().sum(1)
    off = 0.0 if down <= 30 else (dim - 32) * 2.0 ** -39
    want = (inner * 2.0 ** 60 * s * s / (1 + torch.exp(-s)))[:, None]
    rel = 4e-5 + 2.0 ** -8
    spread = 2 * off / s + (off / s) ** 2   # of the square; silu's slope against g / 2 is 1 for small g
    assert ((y - want).abs() <= (rel + (1 + rel) * 1.1 * spread[:, None]) * want).all()
