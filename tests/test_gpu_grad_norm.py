"""GPU parity of the gradients' norm, of clipping and of the clipped AdamW step against the formulas in 64 bits.

Tolerances, derived before the first run, with u = 2^-24 (fp32, half a step): a thread's 32 squares are added in
fp32 with at most 32 roundings in a row, all else in fp64, so the sum is off by 32 u at most, the norm by 16 u, and by
one u more for its own rounding.  The factor: the norm's 16 u and one u.  A clipped gradient: the factor's 17 u and half a
step of its type (fp32 u, bf16 2^-8 of the value; below 2^-126 half of the smallest step, 2^-149 and 2^-133)."""
import math

import numpy as np
import pytest
import torch

from mxfp4_block_scaled_quantize_gb300 import abi
from mxfp4_block_scaled_quantize_gb300.optim import AdamW, GradNorm

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(scope="module", autouse=True)
def _lib():
    import __graft_entry__
    __graft_entry__.build()
    torch.cuda.set_device(0)
    yield
    assert abi.mxfp4_last_device_error() == abi.MXFP4_OK


def f64(t):
    return t.detach().cpu().double().numpy()


def make(sizes, dtype, seed=0, shift=0, scale=1e-3):
    """Gradients of these sizes, each `shift` elements into its storage, between elements of 1e30 that nothing may touch."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    out = []
    for n in sizes:
        store = torch.full((n + shift + 9,), 1e30, dtype=TYPES[dtype], device="cuda")
        g = store[shift:shift + n]
        g.copy_(scale * torch.randn(n, generator=gen, device="cuda"))
        out.append(g)
    return out


def stores(grads):
    return [g.untyped_storage() for g in grads]


def check(grads, dtype, max_norm):
    before = [f64(g) for g in grads]
    kept = [torch.empty(0, dtype=TYPES[dtype], device="cuda").set_(s).clone() for s in stores(grads)]
    norm = math.sqrt(sum(float(np.dot(b, b)) for b in before))
    factor = min(1.0, max_norm / (norm + 1e-6))
    g = GradNorm(grads)
    out = f64(g.measure(grads, max_norm))
    assert abs(out[0] - norm) <= 17 * U * norm
    assert abs(out[1] - factor) <= 17 * U * factor
    again = GradNorm(grads)
    assert np.array_equal(f64(again.measure(grads, max_norm)), out)   # same gradients, same bits
    assert all(torch.equal(k, torch.empty(0, dtype=TYPES[dtype], device="cuda").set_(s)) for k, s in zip(kept, stores(grads)))
    assert np.array_equal(f64(g.clip_(grads, max_norm)), out)
    half = U if dtype == "f32" else 2.0 ** -8
    tiny = 2.0 ** -150 if dtype == "f32" else 2.0 ** -134
    for b, x, k in zip(before, grads, kept):
        want = b * factor
        assert np.all(np.abs(f64(x) - want) <= (half + 18 * U) * np.abs(want) + tiny)
        store = torch.empty(0, dtype=TYPES[dtype], device="cuda").set_(x.untyped_storage())
        first = x.storage_offset()
        assert torch.equal(store[:first], k[:first]) and torch.equal(store[first + x.numel():], k[first + x.numel():])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("sizes, shift", [
    ([1], 0), ([1], 1), ([7, 1, 0, 3], 3), ([8191], 0), ([8192], 0), ([8193], 0), ([8192], 1), ([8185, 8191, 16385], 7),
    ([100003, 5, 65536, 1], 5), ([0, 0, 40], 2), ([3001] * 24, 0)])
def test_norm_and_clipping(dtype, sizes, shift):
    check(make(sizes, dtype, shift=shift), dtype, 0.01)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("count", [48, 49, 1280, 1281, 2561])
def test_lists_of_one_launch_and_more(dtype, count):
    sizes = [1 + (i * 37) % 50 for i in range(count)]
    sizes[count // 2] = 0
    check(make(sizes, dtype, seed=count), dtype, 1e-3)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_more_units_than_ctas(dtype):
    check(make([9000001, 4000003], dtype, shift=1), dtype, 0.5)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("scale", [1e-36, 1e-22, 1e-12, 1e12, 1e19, 1e36])
def test_sizes_whose_squares_leave_fp32(dtype, scale):
    check(make([5000, 33], dtype, scale=scale), dtype, scale)


def test_large_beside_small_and_zeros():
    grads = make([20000, 9000], "f32", scale=1e-25)
    grads[0][777] = 3e25
    grads[1].zero_()
    check(grads, "f32", 1.0)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_no_scaling_below_the_largest_norm(dtype):
    grads = make([10000], dtype)
    kept = grads[0].clone()
    for max_norm in (1e3, math.inf):
        out = GradNorm(grads).clip_(grads, max_norm)
        assert out[1].item() == 1.0 and torch.equal(grads[0], kept)


def test_empty_and_zero():
    grads = make([0, 0], "f32")
    assert GradNorm(grads).clip_(grads, 1.0).tolist() == [0.0, 1.0]
    grads = [torch.zeros(100000, device="cuda")]
    assert GradNorm(grads).measure(grads, 1.0).tolist() == [0.0, 1.0]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_infinities_and_nan(dtype):
    for bad in (math.inf, -math.inf, math.nan):
        grads = make([9000, 50], dtype)
        grads[0][8999] = bad
        norm, factor = GradNorm(grads).clip_(grads, 1.0).tolist()
        if math.isnan(bad):
            assert math.isnan(norm) and math.isnan(factor) and torch.isnan(grads[1]).all()
        else:
            assert norm == math.inf and factor == 0.0
            assert torch.isnan(grads[0][8999]) and not grads[0][:8999].any() and not grads[1].any()


@pytest.mark.parametrize("grad", ["f32", "bf16"])
@pytest.mark.parametrize("bits", [32, 8])
def test_clipped_step_is_the_step_with_the_factor(grad, bits):
    sizes = [3001, 129, 40000]
    gen = torch.Generator(device="cuda").manual_seed(3)
    values = [0.05 * torch.randn(n, generator=gen, device="cuda") for n in sizes]
    grads = make(sizes, grad, scale=0.1)

    def optimizer():
        return AdamW([v.clone() for v in values], state_bits=bits, lr=1e-2)

    clipped, plain = optimizer(), optimizer()
    for t in (1, 2, 3):
        clipped.step(grads, max_norm=0.7, grad_scale=0.5)
        factor = clipped.grad_norm.out[1].item()
        assert 0.0 < factor < 1.0
        # grad_scale times the factor, one rounding in fp32, is what the kernel multiplies by
        plain.step(grads, grad_scale=float(np.float32(0.5) * np.float32(factor)))
        for a, b in zip(clipped.params, plain.params):
            assert torch.equal(a, b)


def test_clipped_step_in_a_graph_with_eager_steps_between():
    sizes = [5000, 77]
    grads = make(sizes, "f32", scale=0.1)
    start = [torch.randn(n, device="cuda") for n in sizes]

    def optimizer():
        return AdamW([v.clone() for v in start], lr=1e-2)

    a, b = optimizer(), optimizer()
    dynamic = torch.empty(4, device="cuda")

    def hyper(t):
        dynamic.copy_(torch.tensor([1e-2, 1 - 0.9 ** t, 1 - 0.999 ** t, 1.0]))

    hyper(1)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):   # its first call is the captured one
        a.step(grads, dynamic=dynamic, max_norm=1.0)
    for t in range(1, 6):
        hyper(t)
        for i, g in enumerate(grads):   # other gradients at the same addresses
            g.copy_(0.1 * t * torch.randn(sizes[i], generator=torch.Generator(device="cuda").manual_seed(t), device="cuda"))
        if t == 3:
            a.step(grads, dynamic=dynamic, max_norm=1.0)
        else:
            graph.replay()
        b.step(grads, dynamic=dynamic, max_norm=1.0)
        assert torch.equal(a.grad_norm.out, b.grad_norm.out)
        assert all(torch.equal(x, y) for x, y in zip(a.params, b.params))


def test_on_a_stream_of_its_own():
    grads = make([300000], "bf16")
    norm = GradNorm(grads)
    want = norm.measure(grads, 1e-3).clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = norm.measure(grads, 1e-3, stream=side)
    side.synchronize()
    assert torch.equal(got, want)
