"""Norm, experts, gradients' norm and update as one run, as a training program and then a server use them."""
import math

import numpy as np
import pytest
import torch

from mxfp4_block_scaled_quantize_gb300 import abi
from mxfp4_block_scaled_quantize_gb300.experts import MXFP4Experts
from mxfp4_block_scaled_quantize_gb300.grouped import MXFP4GroupedLinear
from mxfp4_block_scaled_quantize_gb300.norm import LayerNorm
from mxfp4_block_scaled_quantize_gb300.optim import AdamW, GradNorm

pytestmark = pytest.mark.gpu

T, E, D, N, K = 200, 6, 264, 136, 2   # tokens, experts, width in, width out, experts of a token


@pytest.fixture(scope="module", autouse=True)
def _lib():
    import __graft_entry__
    __graft_entry__.build()
    torch.cuda.set_device(0)
    yield
    assert abi.mxfp4_last_device_error() == abi.MXFP4_OK


class Block:
    """Layer norm, then each token's rows through its experts: weights in bf16 with fp32 masters, the norm's in fp32; one norm
    over all gradients, two optimizers that scale by its factor."""

    def __init__(self, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)

        def rnd(*shape):
            return torch.randn(shape, generator=g, device="cuda")

        self.x = rnd(T, D).to(torch.bfloat16)
        self.target = rnd(T * K, N)
        chosen = torch.rand(T, E, generator=g, device="cuda").topk(K, 1).indices.reshape(-1)
        order = torch.sort(chosen, stable=True).indices
        self.rows = (order // K).to(torch.int32)
        self.offsets = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
        self.offsets[1:] = torch.bincount(chosen, minlength=E).cumsum(0)
        self.master = rnd(E, N, D) * D ** -0.5
        self.w = self.master.to(torch.bfloat16)
        self.gain, self.bias = 1 + 0.1 * rnd(D), 0.1 * rnd(D)
        self.norm = LayerNorm(D, T)
        self.layer = MXFP4GroupedLinear(E, N, D, T * K, out_dtype=torch.float32)
        self.grads_norm = GradNorm([self.w, self.gain, self.bias])
        self.experts_update = AdamW([self.w], masters=[self.master], lr=1e-2)
        self.norm_update = AdamW([self.gain, self.bias], lr=1e-2)
        self.dynamic = torch.empty(4, device="cuda")

    def hyper(self, t):
        self.dynamic.copy_(torch.tensor([1e-2, 1 - 0.9 ** t, 1 - 0.999 ** t, 1.0]))

    def step(self, max_norm):
        h = self.norm.forward(self.x, self.gain, self.bias)
        y = self.layer.forward(h, self.w, self.offsets, self.rows)
        dy = ((y - self.target) * (2 / N)).to(torch.bfloat16)
        dh_rows, dw = self.layer.backward(dy, self.offsets)
        dh = torch.zeros(T, D, device="cuda").index_add_(0, self.rows, dh_rows).to(torch.bfloat16)
        _, dgain, dbias = self.norm.backward(dh, self.x, self.gain)
        grads = [dw, dgain, dbias]
        out = self.grads_norm.measure(grads, max_norm)
        self.experts_update.step(grads[:1], dynamic=self.dynamic, grad_factor=out[1:])
        self.norm_update.step(grads[1:], dynamic=self.dynamic, grad_factor=out[1:])
        return grads, out


def test_a_clipped_step_of_the_whole_block():
    b = Block()
    before = [t.clone() for t in (b.master, b.gain, b.bias)]
    b.hyper(1)
    grads, out = b.step(0.5)
    norm = math.sqrt(sum(float((g.double() ** 2).sum()) for g in grads))
    factor = 0.5 / (norm + 1e-6)
    assert factor < 1 and np.allclose(out.tolist(), [norm, factor], rtol=17 * 2.0 ** -24 * 2)
    for p, old, g in zip((b.master, b.gain, b.bias), before, grads):
        # AdamW's first step: m / c1 = f g, v / c2 = (f g)^2, p = old - lr (f g / (|f g| + 1e-8) + 0.01 old)
        fg = g.double() * factor
        want = old.double() - 1e-2 * (fg / (fg.abs() + 1e-8) + 0.01 * old.double())
        # roundings: of the factor and the product 19 u on f g, which moves f g / (|f g| + 1e-8) by 20 u at most; 30 u for moments,
        # root, quotient and constants of a change below 1e-2 (1 + |old|), 3 u for the difference
        u = 2.0 ** -24
        bound = 50 * u * 1e-2 * (1 + old.double().abs()) + 3 * u * (old.double().abs() + 0.02)
        assert ((p.double() - want).abs() <= bound).all()
    assert torch.equal(b.w, b.master.to(torch.bfloat16))


def test_captured_steps_are_the_eager_ones():
    a, b = Block(3), Block(3)
    a.hyper(1), b.hyper(1)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        a.step(0.5)
    torch.cuda.current_stream().wait_stream(side)
    b.step(0.5)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        a.step(0.5)
    for t in (2, 3, 4):
        a.hyper(t), b.hyper(t)
        graph.replay()
        b.step(0.5)
        # the sum of a token's rows is torch's, of two rows: any order gives the same bits
        for p, q in ((a.master, b.master), (a.w, b.w), (a.gain, b.gain), (a.bias, b.bias), (a.grads_norm.out, b.grads_norm.out)):
            assert torch.equal(p, q)


def test_norm_and_experts_served_in_a_graph():
    dim, inner, experts, top_k = 384, 160, 10, 3
    g = torch.Generator(device="cuda").manual_seed(5)

    def rnd(*shape):
        return torch.randn(shape, generator=g, device="cuda")

    def pack(w):
        return abi.quantize_grouped(w.reshape(-1, w.shape[2]).to(torch.bfloat16), groups=experts, dual=False)[:2]

    up, down = pack(0.05 * rnd(experts, 2 * inner, dim)), pack(0.05 * rnd(experts, dim, inner))
    router, gain, bias = rnd(dim, experts) * dim ** -0.5, 1 + 0.1 * rnd(dim), 0.1 * rnd(dim)
    x = rnd(4, dim).to(torch.bfloat16)

    def serve(norm, layer, x):
        h = norm.forward(x, gain, bias)
        return layer.forward(h, h.float() @ router, *up, *down)

    norm, layer = LayerNorm(dim, 4, train=False), MXFP4Experts(experts, dim, inner, top_k, max_tokens=4)
    eager = LayerNorm(dim, 4, train=False), MXFP4Experts(experts, dim, inner, top_k, max_tokens=4)
    serve(norm, layer, x)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = serve(norm, layer, x)
    for _ in range(4):   # a loop of tokens: the next ones are the outputs
        graph.replay()
        assert torch.equal(y, serve(*eager, x)) and torch.isfinite(y).all() and y.any()
        x.copy_(x + y)
