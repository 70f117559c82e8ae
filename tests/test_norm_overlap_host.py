"""Layer norm's C entries: results that lie where rows are still to be read, without a GPU."""
import pytest

from mxfp4_block_scaled_quantize_gb300 import abi

P, DIM, ROWS = 2 ** 24, 64, 400
BAD = abi.MXFP4_ERR_INVALID_ARG

# x's place and pitch, the result's (in elements from P), rows; is it refused
LAYOUTS = [
    (0, 64, 0, 64, ROWS, False),              # in place
    (0, 70, 0, 70, ROWS, False),
    (0, 64, 0, 70, ROWS, True),               # in place with another pitch
    (0, 64, 0, 70, 1, False),                 # one row has none
    (0, 64, 64, 64, ROWS, True),              # a row further on
    (64, 64, 0, 64, ROWS, True),
    (0, 64, 64 * (ROWS - 1), 64, ROWS, True),
    (0, 64, 64 * ROWS, 64, ROWS, False),      # behind each other
    (64 * ROWS, 64, 0, 64, ROWS, False),
    (0, 64, 8, 64, 1, True),
    (0, 64, 64, 64, 1, False),
    (0, 128, 64, 128, ROWS, False),           # side by side
    (64, 128, 0, 128, ROWS, False),
    (0, 128, 64 + 128 * 3, 128, ROWS, False),
    (0, 128, 63, 128, ROWS, True),
    (0, 128, 65, 128, ROWS, True),            # over the next row's start
    (0, 127, 64, 127, ROWS, True),
    (0, 129, 64, 129, ROWS, False),
    (0, 129, 65, 129, ROWS, False),
    (0, 129, 66, 129, ROWS, True),
    (0, 2 ** 40, 64, 2 ** 40, ROWS, False),
    (0, 2 ** 40, 63, 2 ** 40, ROWS, True),
]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    import __graft_entry__
    __graft_entry__.build()


@pytest.mark.parametrize("flags, size", [(0, 2), (abi.MXFP4_NORM_X_F32, 4)])
@pytest.mark.parametrize("at, pitch, out_at, out_pitch, rows, refused", LAYOUTS)
def test_results_over_rows(at, pitch, out_at, out_pitch, rows, refused, flags, size):
    import torch
    if torch.cuda.is_available():
        pytest.skip("a CUDA device is present: a call that is not refused would run")
    lib = abi.load()
    x, out, apart, v = P + at * size, P + out_at * size, 2 ** 60, 4096
    work, n = 2 ** 61, abi.mxfp4_layer_norm_workspace_bytes(DIM)
    assert (lib.mxfp4_layer_norm(x, rows, DIM, pitch, v, v, 1, 1e-5, flags, out, out_pitch, v, v, None) == BAD) == refused
    for dy, ldy, ax, ldx in ((x, pitch, apart, DIM), (apart, DIM, x, pitch), (x, pitch, x, pitch)):
        status = lib.mxfp4_layer_norm_backward(dy, ldy, ax, rows, DIM, ldx, v, 1, flags, v, v, out, out_pitch, v, v, work, n, None)
        assert (status == BAD) == refused


def test_no_rows_overlap_nothing():
    import torch
    if torch.cuda.is_available():
        pytest.skip("a CUDA device is present: a call that is not refused would run")
    assert abi.load().mxfp4_layer_norm(P, 0, DIM, DIM, None, None, 1, 1e-5, 0, P + 8, DIM, None, None, None) != BAD
