"""GPU parity of the multi-tensor AdamW step against its formula in 64 bits.

Tolerances, derived before the first run, count roundings of u = 2^-24 (fp32, half a step):
  m   two products and a sum, the gradient's scaling: 4 u (|b1 m| + |(1 - b1) g|)
  v   6 u v (one more product)
  p   the difference and the product with lr: 3 u (|p| + |change|), and in change = lr (a + wd p)
      16 u |a| for two corrections, root, quotient and their constants, plus m's error carried
      through a = m / c1 / (sqrt(v / c2) + eps); v's error is inside the 16
  8-bit moments: half an E4M3 step, 2^-4 of the value or 2^-10 of the scale, 2^-9 of it where a
      root is lifted to the smallest code; plus the value's own error and 4 u for the scale.
"""
import numpy as np
import pytest
import torch

from mxfp4_block_scaled_quantize_gb300 import abi
from mxfp4_block_scaled_quantize_gb300.optim import AdamW

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
B = abi.MXFP4_ADAMW_BLOCK


@pytest.fixture(scope="module", autouse=True)
def _lib():
    import __graft_entry__
    __graft_entry__.build()
    torch.cuda.set_device(0)
    yield
    assert abi.mxfp4_last_device_error() == abi.MXFP4_OK


def f64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def decode(codes, scale):
    return f64(codes) * np.repeat(f64(scale), B)[:codes.numel()]


def blocks_max(x):
    pad = np.zeros(-(-x.size // B) * B)
    pad[:x.size] = np.where(np.isfinite(x), np.abs(x), 0.0)
    return pad.reshape(-1, B).max(1)


def reference(p, g, m, v, opt, step, grad_scale=1.0):
    """The step in 64 bits, and the error bounds."""
    (b1, b2), lr, eps, wd = opt.betas, opt.lr, opt.eps, opt.weight_decay
    g = g * grad_scale
    m2, v2 = b1 * m + (1 - b1) * g, b2 * v + (1 - b2) * g * g
    em = 4 * U * (np.abs(b1 * m) + np.abs((1 - b1) * g))
    ev = 6 * U * v2
    c1, c2 = 1 - b1 ** step, 1 - b2 ** step
    denom = np.sqrt(v2 / c2) + eps
    a = m2 / c1 / denom
    change = lr * (a + wd * p)
    ep = 3 * U * (np.abs(p) + np.abs(change)) + lr * (16 * U * np.abs(a) + em / c1 / denom)
    return p - change, m2, v2, ep, em, ev


def make(sizes, param, grad, bits, seed=0, shift=0, scale=1.0):
    """Tensors of these sizes, each `shift` elements into its storage."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dt = {"f32": torch.float32, "bf16": torch.bfloat16}

    def new(n, dtype, values):
        t = torch.zeros(n + shift, dtype=dtype, device="cuda")[shift:]
        t.copy_(values)
        return t

    rnd = lambda n, s: s * torch.randn(n, generator=gen, device="cuda")
    params, masters, grads, m, v = [], [], [], [], []
    for n in sizes:
        w = rnd(n, 0.05)
        params.append(new(n, dt[param.split("_")[0]], w))
        masters.append(new(n, torch.float32, w))
        grads.append(new(n, dt[grad], rnd(n, 1e-2 * scale)))
        m0, r0 = rnd(n, 3e-3 * scale), 1e-2 * scale * torch.rand(n, generator=gen, device="cuda")
        if bits == 32:
            m.append(new(n, torch.float32, m0))
            v.append(new(n, torch.float32, r0 * r0))
        else:
            for out, x in ((m, m0), (v, r0)):
                s = torch.from_numpy(np.maximum(blocks_max(f64(x)) / 448, 2.0 ** -126).astype(np.float32)).cuda()
                y = x / s.repeat_interleave(B)[:n] if n else x
                out.append((new(n, torch.float8_e4m3fn, y.to(torch.float8_e4m3fn)), s))
    opt = AdamW(params, masters=masters if param == "bf16_master" else None, exp_avg=m, exp_avg_sq=v, lr=3e-3,
                betas=(0.9, 0.95), eps=1e-8, weight_decay=0.1)
    return opt, grads


def snapshot(opt):
    source = opt.masters if opt.masters is not None else opt.params
    moments = []
    for m, v in zip(opt.exp_avg, opt.exp_avg_sq):
        moments.append((f64(m), f64(v)) if opt.state_bits == 32 else (decode(*m), decode(*v) ** 2))
    return [f64(p) for p in source], moments


def check_codes(codes, scale, want, err, root, what):
    got_scale, n = f64(scale), want.size
    top = blocks_max(want)
    s = np.maximum(top / 448, 2.0 ** -126)
    assert np.all(np.abs(got_scale - s) <= 4 * U * s + blocks_max(err) / 448), f"{what}: scale"
    s = np.repeat(got_scale, B)[:n]
    y = np.abs(want) / s
    step = np.maximum(2.0 ** -4 * y, 2.0 ** -10)
    if root:
        step = np.where((want > 0) & (y < 2.0 ** -9), 2.0 ** -9, step)
    bound = s * step * (1 + 16 * U) + err * (1 + 2.0 ** -4) + 8 * U * np.abs(want)
    bad = np.abs(decode(codes, scale) - want) > bound
    assert not bad.any(), f"{what}: {bad.sum()} codes off, first {np.argwhere(bad)[0]}"
    if root:
        assert np.all(f64(codes)[want > 0] > 0), f"{what}: a root above zero became zero"


def check_step(opt, before, grads, step, grad_scale=1.0, what=""):
    (p0, moments0) = before
    for j in range(len(opt.params)):
        p, m, v, ep, em, ev = reference(p0[j], f64(grads[j]), *moments0[j], opt, step, grad_scale)
        name = f"{what} tensor {j}"
        if opt.masters is not None:
            assert np.all(np.abs(f64(opt.masters[j]) - p) <= ep), f"{name}: master"
            assert torch.equal(opt.params[j], opt.masters[j].to(torch.bfloat16)), f"{name}: rounding of the master"
        else:
            half = 2.0 ** -8 * np.abs(p) * (1 + 2.0 ** -8) if opt.dtype == torch.bfloat16 else 0.0
            assert np.all(np.abs(f64(opt.params[j]) - p) <= ep + half), f"{name}: parameter"
        if opt.state_bits == 32:
            assert np.all(np.abs(f64(opt.exp_avg[j]) - m) <= em), f"{name}: first moment"
            assert np.all(np.abs(f64(opt.exp_avg_sq[j]) - v) <= ev), f"{name}: second moment"
        else:
            r = np.sqrt(v)
            check_codes(*opt.exp_avg[j], m, em + 2 * U * np.abs(m), False, f"{name}: first moment")
            check_codes(*opt.exp_avg_sq[j], r, 5 * U * r, True, f"{name}: second moment")


SIZES = [1, 7, 8, 127, 128, 129, 0, 1000, 4095, 4096, 4097, 20011]


@pytest.mark.parametrize("shift", [0, 1, 8])
@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("grad", ["f32", "bf16"])
@pytest.mark.parametrize("param", ["f32", "bf16", "bf16_master"])
def test_one_step(param, grad, bits, shift):
    opt, grads = make(SIZES, param, grad, bits, shift=shift)
    before = snapshot(opt)
    opt.step(grads, step=7)
    check_step(opt, before, grads, 7, what=f"{param} {grad} {bits} +{shift}")


@pytest.mark.parametrize("bits", [32, 8])
def test_first_step_from_zero_moments_and_counting(bits):
    p = [torch.randn(300, device="cuda"), torch.randn(5, 40, device="cuda")]
    g = [torch.randn(300, device="cuda"), torch.randn(5, 40, device="cuda")]
    opt = AdamW(p, state_bits=bits)
    for step in (1, 2, 3):
        before = snapshot(opt)
        before = ([x.reshape(-1) for x in before[0]], before[1])
        opt.step(g)
        assert opt.steps == step
        opt.params = [x.view(-1) for x in p]
        check_step(opt, before, [x.view(-1) for x in g], step, what=f"step {step}")


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("count", [40, 41, 320, 700])
def test_many_tensors(count, bits):
    # one table up to 40 tensors, another up to 320, several launches beyond
    opt, grads = make([1 + (i * 37) % 500 for i in range(count)], "bf16_master", "f32", bits, seed=count)
    before = snapshot(opt)
    opt.step(grads, step=3, grad_scale=0.25)
    check_step(opt, before, grads, 3, 0.25, f"{count} tensors")


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("scale", [1e-12, 1e6])
def test_small_and_large_gradients(scale, bits):
    opt, grads = make([513, 4096], "f32", "f32", bits, scale=scale)
    before = snapshot(opt)
    opt.step(grads, step=100)
    check_step(opt, before, grads, 100, what=f"scale {scale}")


def test_zero_gradients_and_zero_moments_only_decay():
    for bits in (32, 8):
        p = torch.randn(200, device="cuda")
        opt = AdamW([p], state_bits=bits, lr=0.1, weight_decay=0.5)
        p0 = f64(p)
        opt.step([torch.zeros(200, device="cuda")])
        assert np.all(np.abs(f64(p) - p0 * 0.95) <= 4 * U * np.abs(p0))
        if bits == 8:
            codes, scale = opt.exp_avg_sq[0]
            assert torch.count_nonzero(codes.view(torch.uint8)) == 0 and f64(scale).tolist() == [2.0 ** -126] * 2


def test_a_large_neighbour_leaves_small_elements_their_direction():
    # one element 2^20 times the others of its block: their roots underflow E4M3's range and take
    # its smallest code, so the next update stays bounded by lr times a few units
    g = torch.full((B,), 1e-6, device="cuda")
    g[5] = 1.0
    p = torch.zeros(B, device="cuda")
    opt = AdamW([p], state_bits=8, lr=1.0, weight_decay=0.0, betas=(0.9, 0.95))
    for _ in range(3):
        opt.step([g])
    assert float(p.abs().max()) <= 3.5
    codes = opt.exp_avg_sq[0][0].float()
    assert bool((codes > 0).all())


@pytest.mark.parametrize("bits", [32, 8])
def test_values_that_are_not_finite_stay_with_their_element(bits):
    n, bad = 384, {3: float("nan"), 130: float("inf"), 300: float("-inf")}
    opt, grads = make([n], "f32", "f32", bits, seed=9)
    clean, same = make([n], "f32", "f32", bits, seed=9)
    for i in bad:
        same[0][i] = 0.0
    for i, x in bad.items():
        grads[0][i] = x
    opt.step(grads, step=2)
    clean.step(same, step=2)
    keep = torch.ones(n, dtype=torch.bool, device="cuda")
    keep[list(bad)] = False
    assert torch.equal(opt.params[0][keep], clean.params[0][keep])
    assert not bool(torch.isfinite(opt.params[0][~keep]).any())
    if bits == 8:
        for (c, _), (d, _) in ((opt.exp_avg[0], clean.exp_avg[0]), (opt.exp_avg_sq[0], clean.exp_avg_sq[0])):
            assert bool(torch.isnan(c.float()[~keep]).all())
            assert bool(torch.isfinite(c.float()[keep]).all())


def test_graph_with_values_on_the_device():
    for bits in (32, 8):
        opt, grads = make([1000, 77], "bf16_master", "bf16", bits, seed=4)
        dynamic = torch.zeros(4, device="cuda")
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            opt.step(grads, step=1, dynamic=dynamic)
        for step in (5, 6):
            b1, b2 = opt.betas
            before = snapshot(opt)
            dynamic.copy_(torch.tensor([opt.lr, 1 - b1 ** step, 1 - b2 ** step, 0.5]))
            graph.replay()
            torch.cuda.synchronize()
            check_step(opt, before, grads, step, 0.5, f"graph {bits} {step}")


def test_another_stream():
    opt, grads = make([5000], "f32", "bf16", 8, seed=6)
    before = snapshot(opt)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        opt.step(grads, step=4)
    s.synchronize()
    check_step(opt, before, grads, 4, what="stream")
