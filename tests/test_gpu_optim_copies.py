"""GPU: an optimizer, a norm and a layer that were copied in the middle of a run go on as the originals do."""
import copy

import pytest
import torch

from mxfp4_block_scaled_quantize_gb300 import abi
from mxfp4_block_scaled_quantize_gb300.norm import LayerNorm
from mxfp4_block_scaled_quantize_gb300.optim import AdamW

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    import __graft_entry__
    __graft_entry__.build()
    torch.cuda.set_device(0)
    yield
    assert abi.mxfp4_last_device_error() == abi.MXFP4_OK


@pytest.mark.parametrize("bits, seed", [(32, None), (8, 5)])
def test_a_copied_optimizer_goes_on_alone(bits, seed):
    gen = torch.Generator(device="cuda").manual_seed(1)

    def rnd():
        return [torch.randn(n, generator=gen, device="cuda") for n in (5000, 77)]

    start = rnd()
    one = AdamW([p.bfloat16() for p in start], masters=[p.clone() for p in start], state_bits=bits, seed=seed)
    grads = [rnd() for _ in range(3)]
    one.step(grads[0], max_norm=1.0)
    two = copy.deepcopy(one)
    kept = [p.clone() for p in one.masters]
    two.step(grads[1], max_norm=1.0)
    assert all(torch.equal(p, k) for p, k in zip(one.masters, kept))   # the original as it was
    one.step(grads[1], max_norm=1.0)
    for a, b in ((one.params, two.params), (one.masters, two.masters), ([one.grad_norm.out], [two.grad_norm.out])):
        assert all(torch.equal(p, q) and p.data_ptr() != q.data_ptr() for p, q in zip(a, b))


def test_a_copied_layer_norm():
    x, w = torch.randn(50, 1000, device="cuda").bfloat16(), torch.randn(1000, device="cuda")
    one = LayerNorm(1000, 50)
    one.forward(x, w, w)
    want = [t.clone() for t in one.backward(x, x, w)]
    two = copy.deepcopy(one)
    two.dw.fill_(9.0), two.db.fill_(9.0)
    assert all(torch.equal(a, b) for a, b in zip(two.backward(x, x, w), want))
