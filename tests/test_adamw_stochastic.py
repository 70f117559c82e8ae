"""Stochastic rounding of AdamW's 8-bit moments: the rule bit for bit, and the recurrences that it
has to follow over many steps.

The rule (restated here in numpy): moments in single fp32 roundings, y = |x| / scale, and the upper
E4M3 neighbour where y's place between the two is at least (r + 1/2) / 2^16, r 16 bits of Philox4x32-10.

Bounds over many steps, derived before their first run.  A code step is at most 1/8 of a value in
E4M3's normal range, and rounding y to a neighbour has a variance of at most (distance to the
nearer grid point) x (code step).  A decay that takes a value to (1 - d) of itself leaves it a
distance d, so its relative variance a step is at most d / 8; over n steps the expected square
grows by (1 + d / 8)^n <= exp(n d / 8) and the expectation stays.  The chance of the upper
neighbour is rounded to 2^-16, half of it a mean error of 2^-17 code steps.
"""
import json
import os

import numpy as np
import pytest
import torch

from mxfp4_block_scaled_quantize_gb300 import abi
from mxfp4_block_scaled_quantize_gb300.optim import AdamW

B = abi.MXFP4_ADAMW_BLOCK
F = np.float32


@pytest.fixture
def gpu():
    import __graft_entry__
    __graft_entry__.build()
    torch.cuda.set_device(0)
    yield
    assert abi.mxfp4_last_device_error() == abi.MXFP4_OK


def philox(counter, key):
    """Philox4x32-10 of counters [..., 4] under one key of two words: [..., 4] words."""
    x = [np.asarray(counter)[..., i].astype(np.uint64) for i in range(4)]
    k, low = [int(w) for w in key], np.uint64(0xFFFFFFFF)
    for _ in range(10):
        a, b = x[0] * np.uint64(0xD2511F53), x[2] * np.uint64(0xCD9E8D57)
        x = [(b >> np.uint64(32)) ^ x[1] ^ np.uint64(k[0]), b & low, (a >> np.uint64(32)) ^ x[3] ^ np.uint64(k[1]), a & low]
        k = [(k[0] + 0x9E3779B9) & 0xFFFFFFFF, (k[1] + 0xBB67AE85) & 0xFFFFFFFF]
    return np.stack(x, axis=-1).astype(np.uint32)


def bits16(n, tensor, step, moment, seed):
    """The 16 bits of each of n elements of a tensor."""
    i = np.arange(-(-n // 8))
    counter = np.stack([i, np.full_like(i, tensor), np.full_like(i, step), np.full_like(i, moment << 31)], axis=-1)
    words = philox(counter, (seed & 0xFFFFFFFF, seed >> 32))
    return np.stack([words & 0xFFFF, words >> 16], axis=-1).reshape(-1)[:n]


def encode(x, root, r):
    """The values of the codes of fp32 x with 16 bits r each, and the scales of its blocks."""
    n, finite = x.size, np.isfinite(x)
    x = np.where(finite, x, F(0))
    pad = np.zeros(-(-n // B) * B, F)
    pad[:n] = np.abs(x)
    scale = np.maximum(pad.reshape(-1, B).max(1) * F(1 / 448), F(2.0 ** -126))
    y = (np.abs(x) / np.repeat(scale, B)[:n]).astype(np.float64)
    grid = 2.0 ** (np.maximum(np.frexp(y)[1] - 1, -6) - 3)
    low = np.floor(y / grid)
    q = np.minimum((low + (y / grid - low >= (r + 0.5) / 65536)) * grid, 448)
    if root:
        q = np.where(x > 0, np.maximum(q, 2.0 ** -9), 0)
    return np.where(finite, np.copysign(q, x), np.nan).astype(F), scale


def test_philox_known_answers():
    with open(os.path.join(os.path.dirname(os.path.abspath(__file__)), "golden", "philox4x32_10_kat.json")) as f:
        for v in json.load(f)["vectors"]:
            ctr, key, out = ([int(w, 16) for w in v[name]] for name in ("ctr", "key", "out"))
            assert philox(np.array(ctr, np.uint64), key).tolist() == out


def test_rounding_is_unbiased():
    # all draws once each (to less than a block): the mean is the value, to half of 2^-16 code steps
    draws = np.arange(65536)[:65536 // (B - 1) * (B - 1)].reshape(-1, B - 1)
    missing = 1 - draws.size / 65536
    for y in (448.0, 447.3, 300.0, 17.0, 16.9, 1.0, 0.99, 2.0 ** -6, 0.7 * 2.0 ** -6, 2.0 ** -9, 0.3 * 2.0 ** -9):
        block = np.append(np.full(B - 1, y, F), F(448))   # the largest makes the scale 1
        q = np.concatenate([encode(block, False, np.append(r, 0))[0][:-1] for r in draws]).astype(np.float64)
        step = 2.0 ** (max(np.frexp(y)[1] - 1, -6) - 3)
        place = float(F(y)) / step
        assert set(np.unique(q / step)) <= {np.floor(place), np.ceil(place)}
        assert abs((q / step).mean() - place) <= 2.0 ** -17 + 2 * missing


def f32(t):
    return t.detach().float().cpu().numpy().astype(F)


def decode(codes, scale):
    return f32(codes) * np.repeat(f32(scale), B)[:codes.numel()]


def make(sizes, grad, seed, betas, shift=0):
    gen = torch.Generator(device="cuda").manual_seed(17)
    params, grads, m, v = [], [], [], []
    for n in sizes:
        params.append(torch.randn(n, generator=gen, device="cuda"))
        g = torch.zeros(n + shift, dtype=grad, device="cuda")[shift:]
        grads.append(g.copy_(1e-2 * torch.randn(n, generator=gen, device="cuda")))
        blocks = -(-n // B)
        for out, signed in ((m, True), (v, False)):
            codes = torch.randint(0, 127, (n,), generator=gen, device="cuda", dtype=torch.int32)
            if signed:
                codes += 128 * torch.randint(0, 2, (n,), generator=gen, device="cuda", dtype=torch.int32)
            store = torch.zeros(n + shift, dtype=torch.uint8, device="cuda")[shift:]
            out.append((store.copy_(codes).view(torch.float8_e4m3fn),
                        1e-5 * (0.5 + torch.rand(blocks, generator=gen, device="cuda"))))
    return AdamW(params, exp_avg=m, exp_avg_sq=v, lr=1e-3, betas=betas, seed=seed), grads


def expected(opt, grads, step, grad_scale=1.0):
    """The moments that a step leaves, per tensor: (m, m_scale), (r, r_scale)."""
    (b1, b2), out, place = opt.betas, [], 0
    for j, g in enumerate(grads):
        if g.numel() == 0:
            out.append(None)
            continue
        gk = f32(g) * F(grad_scale)
        m, r = decode(*opt.exp_avg[j]), decode(*opt.exp_avg_sq[j])
        m = F(b1) * m + F(1 - b1) * gk
        v = F(b2) * (r * r) + F(1 - b2) * gk * gk
        n = g.numel()
        out.append((encode(m, False, bits16(n, place, step, 0, opt.seed)),
                    encode(np.sqrt(v), True, bits16(n, place, step, 1, opt.seed))))
        place += 1
    return out


def check(opt, want, what):
    for j, pair in enumerate(want):
        if pair is None:
            continue
        for (codes, scale), (q, s), name in zip((opt.exp_avg[j], opt.exp_avg_sq[j]), pair, ("first", "second")):
            assert np.array_equal(f32(scale), s), f"{what} tensor {j}: scales of the {name} moment"
            got = f32(codes)
            bad = (got != q) & ~(np.isnan(got) & np.isnan(q))
            assert not bad.any(), f"{what} tensor {j}: {bad.sum()} codes of the {name} moment, first {np.argwhere(bad)[0]}"


@pytest.mark.gpu
@pytest.mark.parametrize("shift", [0, 1, 8])
@pytest.mark.parametrize("grad", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("betas", [(0.9, 0.999), (0.0, 0.5)])
def test_codes_are_the_rules(gpu, betas, grad, shift):
    opt, grads = make([1, 7, 0, 127, 128, 129, 1000, 4096, 20011], grad, (0x9E3779B9 << 32) | 12345, betas, shift)
    for step in (3, 2 ** 24 + 1):
        want = expected(opt, grads, step, 0.5)
        opt.step(grads, step=step, grad_scale=0.5)
        check(opt, want, f"step {step}")


@pytest.mark.gpu
@pytest.mark.parametrize("count", [41, 321, 700])
def test_tensors_are_numbered_through_all_launches(gpu, count):
    opt, grads = make([(i * 37) % 300 for i in range(count)], torch.float32, 5, (0.9, 0.999))
    want = expected(opt, grads, 1)
    opt.step(grads, step=1)
    check(opt, want, f"{count} tensors")


@pytest.mark.gpu
def test_values_that_are_not_finite_become_nan_alone(gpu):
    opt, grads = make([384, 1000], torch.float32, 9, (0.9, 0.999))
    for g in grads:
        g[3], g[130], g[300] = float("nan"), float("inf"), float("-inf")
    want = expected(opt, grads, 2)
    assert all(np.isnan(q).sum() == 3 for pair in want for q, _ in pair)
    opt.step(grads, step=2)
    check(opt, want, "not finite")


@pytest.mark.gpu
def test_a_graph_takes_its_step_from_the_device(gpu):
    opt, grads = make([1000, 77], torch.bfloat16, 21, (0.9, 0.999))
    dynamic = torch.zeros(5, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        opt.step(grads, dynamic=dynamic)
    for step in (5, 6, 6):
        b1, b2 = opt.betas
        want = expected(opt, grads, step)
        dynamic.copy_(torch.tensor([opt.lr, 1 - b1 ** step, 1 - b2 ** step, 1.0, step]))
        graph.replay()
        torch.cuda.synchronize()
        check(opt, want, f"graph {step}")


@pytest.mark.gpu
@pytest.mark.parametrize("moment", ["first", "second"])
def test_decay_keeps_its_expectation(gpu, moment):
    # Half of each block gets no gradient and decays from the block's largest value; the others get
    # gradients of one size, which keep the scale where it is.  First moment: beta1 0.99, d = 0.01,
    # 100 steps; second: beta2 0.999, its root's d = 1 - sqrt(0.999), 2000 steps: n d <= 1.001 in both.
    n, steps, beta = 65536, *((100, 0.99) if moment == "first" else (2000, 0.999))
    decaying = torch.arange(n, device="cuda") % 2 == 1
    p = torch.zeros(n, device="cuda")
    opt = AdamW([p], state_bits=8, lr=0.0, betas=(0.99, 0.999) if moment == "first" else (0.0, 0.999), seed=11)
    (m, m_scale), (v, v_scale) = opt.exp_avg[0], opt.exp_avg_sq[0]
    for t, s in ((m, m_scale), (v, v_scale)):
        t.copy_(torch.full((n,), 448.0, device="cuda"))
        s.fill_(1e-3 / 448)
    g = torch.where(decaying, 0.0, 1e-3)
    for step in range(1, steps + 1):
        opt.step([g], step=step)
    codes, scale = opt.exp_avg[0] if moment == "first" else opt.exp_avg_sq[0]
    got = (codes.double() * scale.double().repeat_interleave(B))[decaying]
    ratio = got / (1e-3 * (beta if moment == "first" else beta ** 0.5) ** steps)
    square = np.exp(1.001 / 8)                          # bound of the expected square
    sigma = np.sqrt((square - 1) / got.numel())         # of the mean
    bias = steps * (2.0 ** -17 / 8 + 8 * 2.0 ** -24)    # of the chances, and of fp32
    assert abs(ratio.mean().item() - 1) <= 6 * sigma + bias
    # of the squares' mean: fourth moments grow by no more than 6 times the variance's exponent, to first order
    assert ratio.square().mean().item() <= square + 6 * np.sqrt((square ** 6 - square ** 2) / got.numel()) + 2 * bias


@pytest.mark.gpu
def test_moments_follow_shrinking_gradients_as_fp32_moments_do(gpu):
    # From step 1000 on every second element's gradients are 100 times smaller: v falls by 10^4, which
    # takes 9200 steps at beta2 = 0.999, and has 2800 more to settle.  Settled, a step moves a root by
    # up to about d = 10^-3 (its own move and its scale's), a relative variance of v of 4 d / 8 a step and
    # of 4 d / 8 / (2 (1 - beta2)) = 0.25 in all: half to twice is two deviations, the median far inside.
    # The update goes with 1 / sqrt(v): a spread of half of v's, which raises its mean square by 0.25 or so.
    # (Codes to nearest: v 7400 times too large, the update 0.01 of what it should be.)
    n = 8192
    gen = torch.Generator(device="cuda").manual_seed(1)
    params = [torch.zeros(n, device="cuda") for _ in range(2)]
    kind = {"betas": (0.9, 0.999), "weight_decay": 0.0, "lr": 1e-3}
    opts = [AdamW([params[0]], state_bits=8, seed=7, **kind), AdamW([params[1]], **kind)]
    small = torch.arange(n, device="cuda") % 2 == 1
    shrink = torch.where(small, 0.01, 1.0)
    moved = torch.zeros(2, 2, device="cuda")   # by moments' type; the small elements, the others
    for t in range(1, 13001):
        g = 1e-3 * torch.randn(n, device="cuda", generator=gen)
        if t > 1000:
            g *= shrink
        for j in (0, 1):
            before = params[j].clone() if t > 12800 else None
            opts[j].step([g])
            if before is not None:
                d = (params[j] - before).square()
                moved[j] += torch.stack([d[small].mean(), d[~small].mean()])
    codes, scale = opts[0].exp_avg_sq[0]
    ratio = (codes.float() * scale.repeat_interleave(B)).square() / opts[1].exp_avg_sq[0]
    for which in (small, ~small):
        assert 0.5 <= ratio[which].median().item() <= 2.0
    for update in (moved[0] / moved[1]).sqrt().tolist():
        assert 0.8 <= update <= 1.4
