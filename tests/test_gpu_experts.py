"""The example of a trained and served layer of experts, and the grouped layer's less common calls."""
import os
import sys

import pytest
import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import experts  # noqa: E402
from mxfp4_block_scaled_quantize_gb300 import abi  # noqa: E402
from mxfp4_block_scaled_quantize_gb300.grouped import MXFP4GroupedLinear  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    import __graft_entry__
    __graft_entry__.build()
    torch.cuda.set_device(0)
    yield
    assert abi.mxfp4_last_device_error() == abi.MXFP4_OK


def test_experts_learn_and_serve():
    losses, router, weight, x = experts.train()
    # The FP4 products' own error is a few percent of the target's variance; half the start is far above it.
    assert losses[-1] < 0.5 * losses[0]
    few = x[:8]
    out = experts.serve(few, router, weight)
    offsets, rows, places, gates = experts.route(few, router, 2)
    layer = MXFP4GroupedLinear(weight.size(0), weight.size(1), weight.size(2), 16, train=False)
    together = experts.gather_outputs(layer.forward(few, weight, offsets, rows), places, gates)
    # The blocks of a token lie along its own row, so its codes do not depend on the batch; the same
    # products are summed in the same K order, so only the gates (a matrix product of another
    # height) may differ: fp32 scores of K terms of size about 1, |gate error| <= K 2^-24 |x||r|.
    bound = 2 * router.size(0) ** 1.5 * 2.0 ** -24 * 16 * together.abs().amax().item() + 2.0 ** -20
    assert (out - together).abs().max().item() <= bound


def _problem(E, sizes, N, K, pitch=0, seed=5):
    g = torch.Generator(device="cuda").manual_seed(seed)
    R = sum(sizes)
    off = torch.tensor([0] + list(torch.tensor(sizes).cumsum(0)), dtype=torch.int32, device="cuda")
    x = torch.randn(R, K + pitch, device="cuda", generator=g).to(torch.bfloat16)
    w = torch.randn(E, N, K, device="cuda", generator=g).to(torch.bfloat16)
    dy = torch.randn(R, N + pitch, device="cuda", generator=g).to(torch.bfloat16)
    return off, x, w, dy


@pytest.mark.parametrize("sizes", [(130, 0, 1, 257), (0, 0, 0, 7), (512, 512, 512, 512)])
def test_pitched_rows_equal_packed_rows(sizes):
    off, x, w, dy = _problem(4, sizes, 264, 328, pitch=24)
    xv, dyv = x[:, :328], dy[:, :264]
    layer = MXFP4GroupedLinear(4, 264, 328, sum(sizes))
    pitched = [t.clone() for t in layer.step(xv, w, dyv, off)]
    packed = layer.step(xv.contiguous(), w, dyv.contiguous(), off)
    for a, b in zip(pitched, packed):
        assert torch.equal(a, b)


@pytest.mark.parametrize("sizes", [(130, 0, 1, 257), (3, 1, 0, 2), (700, 5, 90, 400)])
def test_steps_repeat_bit_for_bit_and_on_another_stream(sizes):
    off, x, w, dy = _problem(4, sizes, 520, 392)
    layer = MXFP4GroupedLinear(4, 520, 392, sum(sizes))
    first = [t.clone() for t in layer.step(x, w, dy, off)]
    for _ in range(4):
        for a, b in zip(first, layer.step(x, w, dy, off)):
            assert torch.equal(a, b)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = layer.step(x, w, dy, off, stream=side.cuda_stream)
    torch.cuda.current_stream().wait_stream(side)
    for a, b in zip(first, other):
        assert torch.equal(a, b)


def test_a_smaller_call_after_a_larger_one():
    off, x, w, dy = _problem(4, (200, 300, 0, 100), 256, 256)
    layer = MXFP4GroupedLinear(4, 256, 256, 600)
    layer.step(x, w, dy, off)
    off2, x2, _, dy2 = _problem(4, (1, 0, 33, 0), 256, 256, seed=6)
    got = [t.clone() for t in layer.step(x2, w, dy2, off2)]
    fresh = MXFP4GroupedLinear(4, 256, 256, 34).step(x2, w, dy2, off2)
    for a, b in zip(got, fresh):
        assert torch.equal(a, b)
    assert not got[2][1].any() and not got[2][3].any()
