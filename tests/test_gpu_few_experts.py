"""GPU parity of the few tokens' layer of experts against its formula in 64 bits.

Tolerances, derived before the first run, with u = 2^-24.  Every product of a code and an activation is exact in fp32.
  c      the sum of a row's products: fp32 with some 32 additions in a block's matrix instructions, which may cut off
         where others round (2 u each), the block's scale, and K / 32 / 16 + 16 blocks after one another: less than 160 u, taken
         as 1e-5 of the sum of magnitudes.  x enters off by 2^-39 of its row's largest at most (fp16's smallest step).
  h      silu(g) u: d(h) = 1.1 |u| d(g) + |silu(g)| d(u) + 12 u |h|; the second product takes h off by 2^-22 |h| + 2^-38 max|h|;
         and 2^-149, where it leaves fp32's range.
  w      a softmax weight: two roundings and expf (2 u) of a difference d of logits: u (|d| + 8), the sum as many: w u (2 max|d| + 24).
  y      sum of w_e (1e-5 sum|W2 h| + sum|W2| d(h)) + d(w_e) |W2 h| + (top_k + 2) u |w_e W2 h|, and half a bf16 step.
"""
import numpy as np
import pytest
import torch

from mxfp4_block_scaled_quantize_gb300 import abi
from mxfp4_block_scaled_quantize_gb300.experts import MXFP4Experts

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
GRID = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])
GRID = np.concatenate([GRID, -GRID])


@pytest.fixture(scope="module", autouse=True)
def _lib():
    import __graft_entry__
    __graft_entry__.build()
    torch.cuda.set_device(0)
    yield
    assert abi.mxfp4_last_device_error() == abi.MXFP4_OK


def f64(t):
    return t.detach().cpu().double().numpy()


def pack(w):
    e, n, k = w.shape
    rows = torch.zeros(e * n, (k + 7) // 8 * 8, dtype=w.dtype, device=w.device)[:, :k]   # the quantizer's pitch is a multiple of 8
    rows.copy_(w.reshape(e * n, k))
    return abi.quantize_grouped(rows, groups=e, dual=False)[:2]


def unpack(blob, e, n, k):
    """The values of expert e's rows, from the layout's definition."""
    q, s = (t.cpu().numpy() for t in blob)
    kp, n_pad = 2 * q.shape[1], -(-n // 128) * 128
    q = q[e * n:(e + 1) * n]
    code = np.stack([q & 15, q >> 4], -1).reshape(n, kp)
    row = e * n_pad + np.arange(n)[:, None]
    b = np.arange(kp // 32)
    byte = s[((row // 128) * (kp // 128) + b // 4) * 512 + (row % 32) * 16 + (row % 128) // 32 * 4 + b % 4]
    return (GRID[code] * np.repeat(2.0 ** (byte.astype(np.float64) - 127), 32, 1))[:, :k]


class Problem:
    def __init__(self, tokens, experts, top_k, dim, inner, seed=0, logits="f32", std=0.05, x_scale=1.0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.sizes = (tokens, experts, top_k, dim, inner)

        def rnd(*shape):
            return torch.randn(shape, generator=g, device="cuda")

        self.x = (x_scale * rnd(tokens, dim)).to(torch.bfloat16)
        self.logits = (2 * rnd(tokens, experts)).to(torch.float32 if logits == "f32" else torch.bfloat16)
        self.up = pack((std * rnd(experts, 2 * inner, dim)).to(torch.bfloat16))
        self.down = pack((std * rnd(experts, dim, inner)).to(torch.bfloat16))

    def layer(self, **kw):
        t, e, k, d, i = self.sizes
        return MXFP4Experts(e, d, i, k, max_tokens=max(1, t), **kw)

    def run(self, layer, x=None, logits=None):
        return layer.forward(self.x if x is None else x, self.logits if logits is None else logits, *self.up, *self.down)

    def want(self, normalize=True, logits=None):
        t, e, k, d, i = self.sizes
        X, L = f64(self.x), f64(self.logits if logits is None else logits)
        y, tol = np.zeros((t, d)), np.zeros((t, d))
        held = {}
        for a in range(t):
            order = sorted(range(e), key=lambda j: (-L[a, j], j))[:k]
            top = L[a, order[0]]
            if top == -np.inf:
                continue
            p = np.exp(L[a, order] - top)
            total = p.sum() if normalize else np.exp(L[a] - top).sum()
            far = max(abs(L[a, j] - top) for j in order if L[a, j] - top > -104)
            for j, pj in zip(order, p):
                if pj < 2.0 ** -150:
                    continue
                if j not in held:
                    held[j] = unpack(self.up, j, 2 * i, d), unpack(self.down, j, d, i)
                up, down = held[j]
                gu = up @ X[a]
                d_gu = 1e-5 * (np.abs(up) @ np.abs(X[a])) + 2.0 ** -39 * np.abs(X[a]).max() * np.abs(up).sum(1)
                g, u = gu[:i], gu[i:]
                with np.errstate(over="ignore"):
                    s = g / (1 + np.exp(-g))
                h = s * u
                dh = 1.1 * np.abs(u) * d_gu[:i] + np.abs(s) * d_gu[i:] + (12 * U + 2.0 ** -22) * np.abs(h) + 2.0 ** -38 * np.abs(h).max(initial=0) + 2.0 ** -149
                out, w = down @ h, pj / total
                y[a] += w * out
                tol[a] += w * (1e-5 * (np.abs(down) @ np.abs(h)) + np.abs(down) @ dh) + \
                    w * U * (2 * far + 24) * np.abs(out) + (k + 2) * U * w * np.abs(out)
        return y, tol

    def check(self, y, normalize=True, logits=None):
        want, tol = self.want(normalize, logits)
        err = np.abs(f64(y) - want)
        bound = tol + 2.0 ** -8 * (np.abs(want) + tol) + 2.0 ** -133
        assert y.shape == want.shape and np.all(err <= bound), np.max(err / bound)


@pytest.mark.parametrize("sizes", [
    (1, 1, 1, 128, 128), (1, 8, 2, 256, 128), (1, 64, 8, 2048, 1408), (2, 3, 3, 1, 1), (3, 5, 2, 33, 31), (5, 7, 2, 1000, 712),
    (8, 16, 4, 512, 384), (9, 16, 4, 512, 384), (13, 7, 2, 1000, 712), (16, 4, 2, 640, 130), (17, 4, 4, 320, 96), (32, 64, 8, 256, 160),
    (40, 2, 2, 384, 256), (64, 8, 3, 136, 200), (64, 64, 6, 384, 320), (64, 300, 16, 130, 66), (7, 1024, 16, 160, 129), (33, 65, 5, 129, 257),
    (2, 2, 1, 7500, 140), (2, 2, 1, 140, 4000), (12, 2, 1, 7400, 60), (12, 2, 1, 60, 3900), (12, 3, 2, 4096, 2048)])
def test_formula(sizes):
    p = Problem(*sizes)
    layer = p.layer()
    y = p.run(layer).clone()
    p.check(y)
    assert torch.equal(p.run(layer), y) and torch.equal(p.run(p.layer()), y)   # the same bits


@pytest.mark.parametrize("logits", ["f32", "bf16"])
@pytest.mark.parametrize("normalize", [True, False])
@pytest.mark.parametrize("tokens", [1, 11, 50])
def test_weights_of_both_kinds(logits, normalize, tokens):
    p = Problem(tokens, 40, 6, 256, 128, seed=3, logits=logits)
    p.check(p.run(p.layer(normalize=normalize)), normalize)


@pytest.mark.parametrize("tokens", [4, 30])
@pytest.mark.parametrize("experts", [6, 70, 257])
def test_equal_logits_go_to_the_lowest_index(tokens, experts):
    p = Problem(tokens, experts, 4, 160, 96, seed=5)
    p.logits.copy_((p.logits * 0.7).round().clamp(-1, 1) * 0.0 + (p.logits > 1))   # zeros and ones
    p.logits[1] = 0.0
    p.logits[2] = -0.0
    p.logits[2, experts // 2:] = 0.0   # the two zeros are equal
    p.check(p.run(p.layer()))


@pytest.mark.parametrize("logits", ["f32", "bf16"])
@pytest.mark.parametrize("tokens", [6, 40])
def test_masks(logits, tokens):
    p = Problem(tokens, 9, 3, 256, 160, seed=7, logits=logits)
    low = torch.finfo(p.logits.dtype).min
    p.logits[:, 4] = low
    p.logits[0] = -float("inf")            # nothing left
    p.logits[1] = low                      # nothing but the type's lowest value: equal logits
    p.logits[2, 2:] = -float("inf")        # fewer experts than choices
    p.logits[3, 1:] = low
    layer = p.layer()
    layer.y.fill_(7.0)
    y = p.run(layer)
    p.check(y)
    assert not y[0].any()
    p.logits[:] = -float("inf")            # a batch of padding alone
    layer.y.fill_(7.0)
    assert not p.run(layer).any()
    p.logits[:] = torch.randn(p.logits.shape, device="cuda")
    p.check(p.run(layer))                  # the counters are as they were


@pytest.mark.parametrize("tokens", [3, 20])
def test_nan_and_infinite_logits(tokens):
    p = Problem(tokens, 12, 3, 256, 128, seed=9)
    clean = p.run(p.layer()).clone()
    p.logits[1, 5] = float("nan")
    p.logits[2, 7] = float("inf")
    y = p.run(p.layer())
    assert torch.isnan(y[1]).all() and torch.isnan(y[2]).all()
    keep = [t for t in range(tokens) if t not in (1, 2)]
    assert torch.equal(y[keep], clean[keep])


@pytest.mark.parametrize("tokens", [3, 20])
def test_nan_and_infinities_in_x_stay_in_their_token(tokens):
    p = Problem(tokens, 12, 3, 256, 128, seed=11)
    clean = p.run(p.layer()).clone()
    p.x[1, 100], p.x[2, 9] = float("nan"), float("inf")
    y = p.run(p.layer())
    assert torch.isnan(y[1]).all() and not torch.isfinite(y[2]).any()
    keep = [t for t in range(tokens) if t not in (1, 2)]
    assert torch.equal(y[keep], clean[keep])


@pytest.mark.parametrize("x_scale, std", [(1e-30, 1.0), (1e30, 2.0 ** -100), (1.0, 2.0 ** -60), (2.0 ** -120, 2.0 ** 40), (1e4, 1.0)])
@pytest.mark.parametrize("tokens", [2, 12])
def test_far_scales(x_scale, std, tokens):
    p = Problem(tokens, 4, 2, 256, 128, seed=13, x_scale=x_scale, std=std)
    p.check(p.run(p.layer()))


def test_one_large_channel_beside_small_ones():
    p = Problem(10, 6, 2, 512, 256, seed=15)
    p.x[:, 7] *= 3e4
    p.x[:, 100:] *= 1e-4
    p.check(p.run(p.layer()))


@pytest.mark.parametrize("tokens", [1, 6, 21])
def test_pitched_and_unaligned_rows(tokens):
    p = Problem(tokens, 10, 3, 264, 136, seed=17)
    want = p.run(p.layer()).clone()
    for at in (8, 3):
        x = torch.full((tokens, 300), 9e9, dtype=torch.bfloat16, device="cuda")[:, at:at + 264]
        x.copy_(p.x)
        logits = torch.full((tokens, 15), 9e9, device="cuda")[:, 2:12]
        logits.copy_(p.logits)
        assert torch.equal(p.run(p.layer(), x, logits), want)


@pytest.mark.parametrize("used", [1, 5, 8, 9])
def test_fewer_tokens_than_the_layer_takes(used):
    p = Problem(20, 10, 3, 256, 128, seed=19)
    layer = p.layer()
    p.run(layer)
    layer.y.fill_(7.0)
    y = layer.forward(p.x[:used], p.logits[:used], *p.up, *p.down)
    assert y.shape == (used, 256) and (layer.y[used:] == 7.0).all()
    part = Problem(20, 10, 3, 256, 128, seed=19)
    part.sizes = (used,) + part.sizes[1:]
    part.x, part.logits = p.x[:used], p.logits[:used]
    part.check(y)
    assert layer.forward(p.x[:0], p.logits[:0], *p.up, *p.down).shape == (0, 256)


def test_a_token_alone_and_in_its_batch():
    p = Problem(8, 10, 3, 256, 128, seed=21)
    layer = p.layer()
    want, tol = p.want()
    for t in range(8):   # the sums' order goes by the batch, the value does not
        err = np.abs(f64(layer.forward(p.x[t:t + 1], p.logits[t:t + 1], *p.up, *p.down)) - want[t:t + 1])
        assert np.all(err <= tol[t] + 2.0 ** -8 * (np.abs(want[t]) + tol[t]))


@pytest.mark.parametrize("tokens", [1, 24])
def test_captured_calls_with_other_inputs(tokens):
    p = Problem(tokens, 16, 4, 512, 256, seed=23)
    layer, plain = p.layer(), p.layer()
    p.run(layer)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        first = p.run(layer).clone()
        second = p.run(layer, x=p.x * 2)
    for seed in (1, 2, 3):
        q = Problem(tokens, 16, 4, 512, 256, seed=seed)
        p.x.copy_(q.x)
        p.logits.copy_(q.logits)
        graph.replay()
        assert torch.equal(first, p.run(plain).clone())
        assert torch.equal(second, p.run(plain, x=p.x * 2))


def test_two_layers_at_once():
    p, q = Problem(20, 16, 4, 512, 256, seed=25), Problem(3, 16, 4, 512, 256, seed=26)
    a, b = p.layer(), q.layer()
    want = p.run(a).clone(), q.run(b).clone()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for _ in range(20):
        for i, (problem, layer) in enumerate(((p, a), (q, b))):
            with torch.cuda.stream(streams[i]):
                got[i].append(problem.run(layer).clone())
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(y, want[i]) for y in got[i])


def test_many_calls_in_a_row():
    p = Problem(1, 32, 8, 640, 320, seed=27)
    layer = p.layer()
    outs = []
    for t in range(50):
        logits = torch.roll(p.logits, t, 1)
        outs.append((logits, p.run(layer, logits=logits).clone()))
    for logits, y in outs[::7]:
        p.check(y, logits=logits)
