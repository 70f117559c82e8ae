"""GPU parity of layer norm and its backward pass against the formulas in 64 bits.

Tolerances, derived before the first run.  u = 2^-24, n elements a row, s their deviation, r = 1 / sqrt(s^2 + eps),
xh = (x - mu) r.  A row's sum is at most 32 additions in a thread and 10 across them: depth D = 45.
  mean   the first one is off by D u mean|x|; the centred values' own sum corrects it, off by (D + 1) u mean|x - mu|,
         and it is rounded once: u |mu| + 50 u s
  r      the sum of squares is off by (D + 3) u, its root by half of that, root and quotient by 3 u: 30 u
  xh     d(xh) = u (34 |xh| + 52 + 2 |mu| r)
  y      |g| d(xh) + 2 u (|g xh| + |b|) + half a step of its type
  dx     a = dy g, A = mean|a|, B = mean|a xh|:  r [6 u |a| + (D + 4) u A + |xh| ((D + 6) u B + mean(|a| d(xh))) + d(xh) |mean(a xh)|]
         + 31 u |dx| + half a step
  dw, db sums over R rows in some order: (R + 64) u of the sum of magnitudes, in dw plus sum |dy| d(xh)
"""
import numpy as np
import pytest
import torch

from mxfp4_block_scaled_quantize_gb300 import abi
from mxfp4_block_scaled_quantize_gb300.norm import LayerNorm

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HALF = {torch.float32: (U, 2.0 ** -149), torch.bfloat16: (2.0 ** -8, 2.0 ** -133)}


@pytest.fixture(scope="module", autouse=True)
def _lib():
    import __graft_entry__
    __graft_entry__.build()
    torch.cuda.set_device(0)
    yield
    assert abi.mxfp4_last_device_error() == abi.MXFP4_OK


def f64(t):
    return t.detach().cpu().double().numpy()


def within(got, want, tol, dtype, what):
    half, tiny = HALF[dtype]
    err = np.abs(f64(got) - want)
    bound = tol + half * (np.abs(want) + tol) + tiny
    assert got.shape == want.shape and np.all(err <= bound), f"{what}: {np.max(err / bound)} of the bound"


def make(rows, dim, dtype, w_dtype, samples, pitch=0, seed=0, mean=0.5, std=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def rnd(*shape):
        return torch.randn(shape, generator=g, device="cuda")

    x = torch.full((rows, dim + pitch), 7e4, dtype=dtype, device="cuda")[:, :dim]
    x.copy_(std * rnd(rows, dim) * (1 + 15 * (rnd(dim) > 2)) + mean * rnd(rows, 1))
    dy = torch.full((rows, dim + pitch), 7e4, dtype=dtype, device="cuda")[:, :dim]
    dy.copy_(1e-2 * rnd(rows, dim))
    w = b = None
    if w_dtype is not None:
        shape = (dim,) if samples is None else (samples, dim)
        w, b = (1 + 0.3 * rnd(*shape)).to(w_dtype), (0.3 * rnd(*shape)).to(w_dtype)
    return x, dy, w, b


def formulas(x, dy, w, b, eps, add_one):
    X, DY = f64(x), f64(dy)
    R = X.shape[0]

    def spread(v, none):
        if v is None:
            return np.full_like(X, none)
        v = f64(v).reshape(-1, X.shape[1])
        return np.repeat(v, R // v.shape[0], 0)

    g, bias = spread(w, 1.0), spread(b, 0.0)
    if add_one and w is not None:
        g = g + 1
    mu = X.mean(1, keepdims=True)
    r = 1 / np.sqrt(((X - mu) ** 2).mean(1, keepdims=True) + eps)
    xh = (X - mu) * r
    dxh = U * (34 * np.abs(xh) + 52 + 2 * np.abs(mu) * r)
    y, y_tol = xh * g + bias, np.abs(g) * dxh + 2 * U * (np.abs(g * xh) + np.abs(bias))
    a = DY * g
    m2 = (a * xh).mean(1, keepdims=True)
    dx = r * (a - a.mean(1, keepdims=True) - xh * m2)
    A, B = np.abs(a).mean(1, keepdims=True), np.abs(a * xh).mean(1, keepdims=True)
    dx_tol = r * (6 * U * np.abs(a) + 49 * U * A + np.abs(xh) * (51 * U * B + (np.abs(a) * dxh).mean(1, keepdims=True)) +
                  dxh * np.abs(m2)) + 31 * U * np.abs(dx)
    S = 1 if w is None or w.dim() == 1 else w.shape[0]

    def sums(v):
        return v.reshape(S, R // S, -1).sum(1)

    dw, db = sums(DY * xh), sums(DY)
    dw_tol = (R // S + 64) * U * sums(np.abs(DY * xh)) + sums(np.abs(DY) * dxh)
    db_tol = (R // S + 64) * U * sums(np.abs(DY))
    shape = (X.shape[1],) if w is None else tuple(w.shape)
    return y, y_tol, dx, dx_tol, dw.reshape(shape), dw_tol.reshape(shape), db.reshape(shape), db_tol.reshape(shape)


def check(rows, dim, dtype=torch.bfloat16, w_dtype=torch.float32, samples=None, pitch=0, add_one=False, eps=1e-5, **kind):
    x, dy, w, b = make(rows, dim, dtype, w_dtype, samples, pitch, **kind)
    layer = LayerNorm(dim, rows + 3, eps=eps, dtype=dtype, add_one=add_one, max_samples=samples or 1)
    for t in (layer.y, layer.dx):
        t.fill_(9.0)
    for t in (layer.dw, layer.db):
        t.fill_(9.0)
    y = layer.forward(x, w, b)
    dx, dw, db = layer.backward(dy, x, w)
    want = formulas(x, dy, w, b, eps, add_one)
    within(y, *want[0:2], dtype, "y")
    within(dx, *want[2:4], dtype, "dx")
    if w is None:
        assert dw is None and db is None
    else:
        within(dw, *want[4:6], torch.float32, "dw")
        within(db, *want[6:8], torch.float32, "db")
    assert (layer.y[rows:] == 9.0).all() and (layer.dx[rows:] == 9.0).all()   # rows behind the last stay as they were
    if w is None:
        assert (layer.dw == 9.0).all() and (layer.db == 9.0).all()
    kept = [t.clone() for t in (y, dx) + (() if w is None else (dw, db))]
    layer.forward(x, w, b)
    again = [t for t in (layer.y[:rows],) + layer.backward(dy, x, w) if t is not None]
    assert all(torch.equal(p, q) for p, q in zip(kept, again))   # the same bits
    serving = LayerNorm(dim, rows, eps=eps, dtype=dtype, add_one=add_one, max_samples=samples or 1, train=False)
    assert torch.equal(serving.forward(x, w, b), kept[0])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("dim", [1, 2, 7, 8, 31, 32, 33, 128, 255, 256, 257, 264, 512, 520, 1000, 1001, 1024, 1025, 1032, 2048, 4096, 4097,
                                 4104, 5120, 8192, 8193, 8200, 16383, 16384])
def test_every_width(dtype, dim):
    check(5, dim, dtype)


@pytest.mark.parametrize("rows", [1, 2, 7, 8, 9, 303, 304, 305, 609, 2433, 5000])
@pytest.mark.parametrize("dim", [72, 333, 1000, 1544])
def test_every_number_of_rows(rows, dim):
    check(rows, dim)


@pytest.mark.parametrize("rows, dim, samples, dtype", [(4900, 4104, 1, torch.bfloat16), (2574, 4608, 78, torch.bfloat16), (2541, 5120, 77, torch.float32)])
def test_many_rows_of_a_cta(rows, dim, samples, dtype):
    check(rows, dim, dtype, torch.float32, samples)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("w_dtype", [None, torch.bfloat16, torch.float32])
@pytest.mark.parametrize("dim, pitch", [(256, 8), (256, 3), (1100, 0), (1104, 16), (2304, 1)])
def test_types_and_pitches(dtype, w_dtype, dim, pitch):
    check(37, dim, dtype, w_dtype, pitch=pitch)


@pytest.mark.parametrize("w_dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows, dim, samples", [(6, 128, 2), (1000, 1104, 2), (999, 333, 3), (64, 2048, 64), (400, 77, 400), (3000, 264, 600),
                                                (610, 1032, 305), (4, 264, 1)])
def test_vectors_of_samples(w_dtype, rows, dim, samples):
    check(rows, dim, w_dtype=w_dtype, samples=samples, add_one=True)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows, dim, samples", [(1, 1001, 1), (2, 333, 1), (3, 2501, 1), (7, 1003, 1), (8, 505, 1), (9, 4100, 1), (4200, 1003, 1), (4300, 1541, 2), (700, 8191, 7), (17, 250, 1),
                                                (100, 8191, 1), (640, 2050, 2), (1300, 517, 5), (3000, 1005, 600), (2000, 70, 500)])
def test_rows_that_start_anywhere(dtype, rows, dim, samples):
    check(rows, dim, dtype, samples=None if samples == 1 else samples)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("dim", [260, 1001, 2300])
@pytest.mark.parametrize("at_x, at_dy", [(1, 1), (3, 3), (1, 2), (0, 5), (8, 8)])
def test_tensors_shifted_alike_and_not(dtype, dim, at_x, at_dy):
    x, dy, w, b = make(40, dim, dtype, torch.float32, None, seed=8)

    def moved(t, at):
        store = torch.full((40 * (dim + 3) + at,), 7e4, dtype=dtype, device="cuda")
        view = store[at:].view(40, dim + 3)[:, :dim]
        view.copy_(t)
        return view

    layer = LayerNorm(dim, 40, dtype=dtype)
    xv, dyv = moved(x, at_x), moved(dy, at_dy)
    y = layer.forward(xv, w, b)
    dx, dw, db = layer.backward(dyv, xv, w)
    want = formulas(x, dy, w, b, 1e-5, False)
    within(y, *want[0:2], dtype, "y")
    within(dx, *want[2:4], dtype, "dx")
    within(dw, *want[4:6], torch.float32, "dw")
    within(db, *want[6:8], torch.float32, "db")


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("dim", [100, 1536])
def test_a_mean_far_above_the_deviation(dtype, dim):
    check(50, dim, dtype, mean=300.0, std=0.01 if dtype == torch.float32 else 1.0)


def test_constant_rows_and_zeros():
    x = torch.zeros(4, 1536, device="cuda")
    x[1] = 3.25
    x[2] = -1e6
    layer = LayerNorm(1536, 4, dtype=torch.float32)
    b = torch.randn(1536, device="cuda")
    y = layer.forward(x, torch.randn(1536, device="cuda"), b)
    assert torch.equal(y, b.expand(4, -1))   # nothing but the bias


def test_views_inside_a_larger_tensor_and_unaligned_vectors():
    store = torch.randn(20, 3 * 256, device="cuda").to(torch.bfloat16)
    for at in (256, 255):
        x = store[:, at:at + 256]
        w = torch.randn(257, device="cuda")[1:]
        layer, other = LayerNorm(256, 20), LayerNorm(256, 20)
        # sums in another order, so values some 2^-20 apart before they are rounded: one step of bf16, 2^-7, at most
        assert torch.allclose(layer.forward(x, w).float(), other.forward(x.contiguous(), w.clone()).float(), rtol=2.0 ** -7, atol=1e-5)
        dy = store[:, :256]
        for p, q in zip(layer.backward(dy, x, w)[:2], other.backward(dy.contiguous(), x.contiguous(), w.clone())[:2]):
            assert torch.allclose(p.float(), q.float(), rtol=2.0 ** -7, atol=1e-5)   # sums in another order: one rounding of bf16 apart


def test_infinities_stay_in_their_rows():
    x = torch.randn(6, 1032, device="cuda").to(torch.bfloat16)
    clean = LayerNorm(1032, 6).forward(x).clone()
    x[2, 5], x[4, 7] = float("inf"), float("nan")
    y = LayerNorm(1032, 6).forward(x)
    for i in range(6):
        assert torch.isnan(y[i]).all() if i in (2, 4) else torch.equal(y[i], clean[i])


@pytest.mark.parametrize("samples", [None, 2])
def test_no_rows(samples):
    layer = LayerNorm(64, 0, max_samples=2)
    x = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda")
    w = torch.ones((64,) if samples is None else (samples, 64), device="cuda")
    assert layer.forward(x, w, w).shape == (0, 64)
    dx, dw, db = layer.backward(x, x, w)
    assert dx.shape == (0, 64) and not dw.any() and not db.any()


def test_gradient_against_differences():
    # central differences of a loss in 64 bits, the layer in fp32: the loss's third derivative at step h leaves about h^2
    x, dy, w, b = make(3, 40, torch.float32, torch.float32, None, seed=4)
    layer = LayerNorm(40, 3, dtype=torch.float32)
    layer.forward(x, w, b)
    dx, dw, db = layer.backward(dy, x, w)

    def loss(x, w, b):
        mu = x.mean(1, keepdim=True)
        return (((x - mu) / torch.sqrt(((x - mu) ** 2).mean(1, keepdim=True) + 1e-5) * w + b) * dy.double()).sum().item()

    values = [t.double() for t in (x, w, b)]
    h = 1e-4
    for which, grad in enumerate((dx, dw, db)):
        for i in range(0, values[which].numel(), 7):
            up, down = ([v.clone() for v in values] for _ in range(2))
            up[which].view(-1)[i] += h
            down[which].view(-1)[i] -= h
            slope = (loss(*up) - loss(*down)) / (2 * h)
            assert abs(slope - grad.reshape(-1)[i].item()) <= 1e-6 + 1e-4 * abs(slope)


def test_captured_step_with_other_inputs():
    x, dy, w, b = make(500, 1544, torch.bfloat16, torch.float32, None)
    layer, plain = LayerNorm(1544, 500), LayerNorm(1544, 500)
    layer.forward(x, w, b)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = layer.forward(x, w, b)
        grads = layer.backward(dy, x, w)
    for seed in (1, 2):
        for t, v in zip((x, dy, w, b), make(500, 1544, torch.bfloat16, torch.float32, None, seed=seed)):
            t.copy_(v)
        graph.replay()
        assert torch.equal(y, plain.forward(x, w, b))
        assert all(torch.equal(p, q) for p, q in zip(grads, plain.backward(dy, x, w)))


def test_rows_beyond_32_bits_of_elements():
    # 2^31 elements and more between the first row and the last
    rows, dim = 5, 64
    store = torch.empty(4 * 2 ** 29 + 64, dtype=torch.bfloat16, device="cuda")
    x = store.as_strided((rows, dim), (2 ** 29, 1))
    v = torch.randn(rows, dim, device="cuda").to(torch.bfloat16)
    x.copy_(v)
    layer, plain = LayerNorm(dim, rows), LayerNorm(dim, rows)
    assert torch.equal(layer.forward(x), plain.forward(v))
    assert torch.equal(layer.backward(x, x)[0], plain.backward(v, v)[0])
