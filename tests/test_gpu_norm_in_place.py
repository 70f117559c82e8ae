"""GPU: layer norm whose results take the place of its rows, or lie beside them."""
import pytest
import torch

from mxfp4_block_scaled_quantize_gb300 import abi
from mxfp4_block_scaled_quantize_gb300.norm import LayerNorm

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    import __graft_entry__
    __graft_entry__.build()
    torch.cuda.set_device(0)
    yield
    assert abi.mxfp4_last_device_error() == abi.MXFP4_OK


def run(x, dy, w, y, dx):
    """The C entries into y and dx: y as it was after the forward pass, dx, dw."""
    rows, dim = x.shape
    flags = (abi.MXFP4_NORM_X_F32 if x.dtype == torch.float32 else 0) | abi.MXFP4_NORM_W_F32
    mean, rstd, dw = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda"), torch.empty(dim, device="cuda")
    work = torch.empty(abi.mxfp4_layer_norm_workspace_bytes(dim), dtype=torch.uint8, device="cuda")
    kept = x.clone()
    abi.mxfp4_layer_norm(x, rows, dim, x.stride(0), w, None, 1, 1e-5, flags, y, y.stride(0), mean, rstd)
    out = y.clone()
    x.copy_(kept)   # where y was x
    abi.mxfp4_layer_norm_backward(dy, dy.stride(0), x, rows, dim, x.stride(0), w, 1, flags, mean, rstd, dx, dx.stride(0), dw, None, work, work.numel())
    return out, dx.clone(), dw


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("dim", [64, 333, 1000, 1001, 4100, 4104, 5120, 8200])
@pytest.mark.parametrize("rows", [1, 7, 3000])
def test_in_place_gives_the_same_bits(dtype, dim, rows):
    def make(seed):
        return torch.randn(rows, dim, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda").to(dtype)

    w = torch.randn(dim, device="cuda")
    want = run(make(1), make(2), w, torch.empty(rows, dim, dtype=dtype, device="cuda"), torch.empty(rows, dim, dtype=dtype, device="cuda"))
    for place in ("x", "dy"):
        x, dy = make(1), make(2)
        got = run(x, dy, w, x, x if place == "x" else dy)
        assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("dim", [64, 333, 1001, 1024])
def test_side_by_side(dtype, dim):
    rows = 900
    store = torch.randn(rows, 3 * dim, device="cuda").to(dtype)
    x, dy, out = store[:, :dim], store[:, dim:2 * dim], store[:, 2 * dim:]
    w = torch.randn(dim, device="cuda")
    # the same places, so the same accesses and the same order of sums
    other = store.clone()
    apart = torch.empty_like(store)[:, 2 * dim:]
    want = run(other[:, :dim], other[:, dim:2 * dim], w, apart, apart)
    got = run(x, dy, w, out, out)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert torch.equal(store[:, :2 * dim], other[:, :2 * dim])


def test_a_layer_takes_its_own_result_but_not_a_row_further():
    layer, other = LayerNorm(1000, 40), LayerNorm(1000, 40)
    x = torch.randn(40, 1000, device="cuda").to(torch.bfloat16)
    y = layer.forward(x)
    want = other.forward(y.clone()).clone()
    assert torch.equal(layer.forward(y), want)
    for bad in (layer.y[1:], layer.y.view(-1)[8:8 + 39 * 1000].view(39, 1000)):
        with pytest.raises(abi.Mxfp4Error):
            layer.forward(bad)
    layer.forward(x[:39])
    with pytest.raises(abi.Mxfp4Error):
        layer.backward(layer.dx[1:], x[:39])
