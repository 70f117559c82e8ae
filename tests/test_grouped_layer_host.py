"""Refusals of the grouped layer that need no GPU: the order of its calls and what it is handed."""
import pytest
import torch

from mxfp4_block_scaled_quantize_gb300 import abi
from mxfp4_block_scaled_quantize_gb300.grouped import MXFP4GroupedLinear

E, N, K, R = 2, 8, 24, 10


@pytest.fixture(scope="module", autouse=True)
def _lib():
    import __graft_entry__
    __graft_entry__.build()


@pytest.fixture
def calls(monkeypatch):
    """The library's calls, noted instead of made; the host stands in for the layer's GPU."""
    made = []
    monkeypatch.setattr(MXFP4GroupedLinear, "_here", staticmethod(lambda t: t.get_device()))
    for name in ("mxfp4_quantize_grouped", "mxfp4_grouped_forward", "mxfp4_grouped_backward"):
        monkeypatch.setattr(abi, name, lambda *a, _name=name, **k: made.append((_name, a)))
    return made


def layer(train=True):
    return MXFP4GroupedLinear(E, N, K, R, train=train, device="cpu")


def bf16(*shape):
    return torch.zeros(shape, dtype=torch.bfloat16)


OFFSETS = torch.zeros(E + 1, dtype=torch.int32)


@pytest.mark.parametrize("train", [True, False])
def test_products_need_weights_that_were_quantized(train, calls):
    ours = layer(train)
    with pytest.raises(ValueError, match="no weights quantized"):
        ours.forward(bf16(4, K), None, OFFSETS)
    assert not calls
    ours.quantize_w(bf16(E, N, K))
    ours.forward(bf16(4, K), None, OFFSETS)
    ours = layer(train)
    ours.forward(bf16(4, K), bf16(E, N, K), OFFSETS)   # quantizes them too
    ours.forward(bf16(4, K), None, OFFSETS)


def test_packed_weights_have_no_gradient(calls):
    # dX comes from the col blob of W, which packed weights do not have
    ours = layer()
    w_q, w_s = abi.alloc_grouped_blobs(E * N, K, E, equal=True, dual=False, device="cpu")
    ours.forward(bf16(4, K), bf16(E, N, K), OFFSETS)
    ours.forward_packed(bf16(4, K), w_q, w_s, OFFSETS)
    with pytest.raises(ValueError, match="packed"):
        ours.backward(bf16(4, N), OFFSETS)
    assert "mxfp4_grouped_backward" not in [name for name, _ in calls]
    ours.forward(bf16(4, K), None, OFFSETS)
    ours.backward(bf16(4, N), OFFSETS)


def test_backward_takes_the_rows_of_its_forward(calls):
    # the row count sets the pitch of X's col blob
    ours = layer()
    with pytest.raises(ValueError, match="forward"):
        ours.backward(bf16(4, N), OFFSETS)
    ours.forward(bf16(6, K), bf16(E, N, K), OFFSETS)
    for rows in (5, 7, 0):
        with pytest.raises(ValueError, match="6 rows"):
            ours.backward(bf16(rows, N), OFFSETS)
    assert "mxfp4_grouped_backward" not in [name for name, _ in calls]
    ours.backward(bf16(6, N), OFFSETS)
    ours.forward(bf16(3, K), None, OFFSETS, torch.zeros(7, dtype=torch.int32))   # gathered: 7 rows
    with pytest.raises(ValueError, match="7 rows"):
        ours.backward(bf16(6, N), OFFSETS)
    ours.backward(bf16(7, N), OFFSETS)


@pytest.mark.parametrize("train", [True, False])
def test_packed_weights_of_another_layout_are_refused(train, calls):
    # the blob's extents come from E, N and K alone: a shorter one would be read past its end
    ours = layer(train)
    w_q, w_s = abi.alloc_grouped_blobs(E * N, K, E, equal=True, dual=False, device="cpu")
    strided_q, strided_s = w_q.repeat(1, 2)[:, ::2], w_s.repeat(2)[::2]
    for q, s in ((w_q[:-1], w_s), (w_q[:, :K // 2].contiguous(), w_s), (w_q, w_s[:-1]), (strided_q, w_s),
                 (w_q, strided_s), (w_q.float(), w_s), (w_q, w_s.short()), (None, w_s), (w_q, None),
                 (w_q.data_ptr(), w_s)):
        with pytest.raises(ValueError, match="packed weights"):
            ours.forward_packed(bf16(4, K), q, s, OFFSETS)
    assert not calls
    ours.forward_packed(bf16(4, K), w_q, w_s, OFFSETS)
    ours.forward_packed(bf16(4, K), w_q.view(E, N, -1), w_s.view(torch.int8), OFFSETS)   # any view of the same bytes


def test_tensors_elsewhere_are_refused():
    # a host address would be dereferenced on the GPU
    for ours in (layer(True), layer(False)):
        w_q, w_s = abi.alloc_grouped_blobs(E * N, K, E, equal=True, dual=False, device="cpu")
        with pytest.raises(ValueError, match="GPU"):
            ours.quantize_w(bf16(E, N, K))
        with pytest.raises(ValueError, match="GPU"):
            ours.forward(bf16(4, K), bf16(E, N, K), OFFSETS)
        with pytest.raises(ValueError, match="GPU"):
            ours.forward_packed(bf16(4, K), w_q, w_s, OFFSETS)


@pytest.mark.parametrize("which", ["x", "w", "offsets", "rows", "dy", "backward's offsets", "w_q", "w_s"])
def test_each_tensor_is_on_the_layers_device(which, calls):
    class OnAnotherGpu(torch.Tensor):
        def get_device(self):
            return 1

    ours = layer()
    t = {"x": bf16(4, K), "w": bf16(E, N, K), "offsets": OFFSETS, "rows": torch.zeros(4, dtype=torch.int32),
         "dy": bf16(4, N), "backward's offsets": OFFSETS}
    t["w_q"], t["w_s"] = abi.alloc_grouped_blobs(E * N, K, E, equal=True, dual=False, device="cpu")
    ok = dict(t)
    t[which] = t[which].as_subclass(OnAnotherGpu)
    if which in ("dy", "backward's offsets"):
        ours.forward(ok["x"], ok["w"], ok["offsets"], ok["rows"])
        call = lambda t: ours.backward(t["dy"], t["backward's offsets"])
    elif which in ("w_q", "w_s"):
        call = lambda t: ours.forward_packed(t["x"], t["w_q"], t["w_s"], t["offsets"], t["rows"])
    else:
        call = lambda t: ours.forward(t["x"], t["w"], t["offsets"], t["rows"])
    made = len(calls)
    with pytest.raises(ValueError, match="GPU"):
        call(t)
    assert len(calls) == made
    call(ok)
    if which == "w":
        with pytest.raises(ValueError, match="GPU"):
            ours.quantize_w(t["w"])


def test_grouped_quantizer_takes_gpu_tensors_only(calls):
    x = bf16(4, K)
    for args in ((x, OFFSETS), (x, None, None, 2)):
        with pytest.raises(ValueError, match="GPU"):
            abi.quantize_grouped(*args)
    assert not calls


def test_weights_quantized_after_the_forward_are_not_its_weights(calls):
    # they replace the blobs that the forward used, so dX would be another W's
    ours = layer()
    ours.forward(bf16(4, K), bf16(E, N, K), OFFSETS)
    ours.quantize_w(bf16(E, N, K))
    with pytest.raises(ValueError, match="no forward"):
        ours.backward(bf16(4, N), OFFSETS)
    ours.forward(bf16(4, K), None, OFFSETS)
    ours.backward(bf16(4, N), OFFSETS)


def test_one_row_has_no_pitch(calls):
    # the stride of an axis of one element means nothing: a column turned round is one whole row
    ours = layer()
    row = bf16(K, 1).t()
    assert row.stride() == (1, 1) and row.is_contiguous()
    ours.forward(row, bf16(E, N, K), OFFSETS)
    ours.backward(bf16(N, 1).t(), OFFSETS)
    for name, args in calls:
        ld, k = {"mxfp4_grouped_forward": (args[3], K), "mxfp4_grouped_backward": (args[2], N)}[name]
        assert ld >= k and ld % 8 == 0


def test_one_row_has_no_pitch_in_the_quantizer(calls, monkeypatch):
    class Row(torch.Tensor):
        is_cuda = True

    monkeypatch.setattr(abi, "alloc_grouped_blobs", lambda *a: (None,) * 4)
    abi.quantize_grouped(bf16(20, 1).t().as_subclass(Row), None, None, 1)
    (_, args), = calls
    assert args[3] >= 20 and args[3] % 8 == 0


def test_forwards_with_own_and_packed_weights_in_turn(calls):
    # each call's weights are the ones it was given, and a refused call changes nothing for the backward
    ours = layer()
    own = [b.data_ptr() for b in ours.w_blobs]
    w_q, w_s = abi.alloc_grouped_blobs(E * N, K, E, equal=True, dual=False, device="cpu")
    seen = []

    def note():
        seen.append(list(calls[-1][1][0].w_blobs[:2]))

    ours.forward(bf16(4, K), bf16(E, N, K), OFFSETS)
    note()
    with pytest.raises(ValueError):
        ours.forward_packed(bf16(4, K), w_q, w_s, OFFSETS[:-1])
    ours.backward(bf16(4, N), OFFSETS)
    assert list(calls[-1][1][0].w_blobs[2:]) == own[2:]
    ours.forward(bf16(4, K), None, OFFSETS)
    note()
    ours.forward_packed(bf16(4, K), w_q, w_s, OFFSETS)
    note()
    ours.forward(bf16(4, K), bf16(E, N, K), OFFSETS)
    note()
    assert seen == [own[:2], own[:2], [w_q.data_ptr(), w_s.data_ptr()], own[:2]]
