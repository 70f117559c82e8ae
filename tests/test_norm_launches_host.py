"""How layer norm's backward pass shares out its rows and where the partial rows of dw and db go, by the library's own C entry with its
launches noted, without a GPU."""
import ctypes
import os
import subprocess

import pytest

from mxfp4_block_scaled_quantize_gb300 import abi, build

HERE = os.path.dirname(os.path.abspath(__file__))
NAMES = ("ctas", "chunks", "chunk_rows", "sample_rows", "period", "access", "partial_w", "partial_b", "reduced", "reduced_chunks", "reduced_samples")
DW, DB, WORKSPACE = 2 ** 40, 2 ** 41, 2 ** 44
SHIFTED = 2   # the access of rows that start anywhere, in groups of 16 bytes


class Noted(ctypes.Structure):
    _fields_ = [(name, ctypes.c_int64) for name in NAMES]


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    out = str(tmp_path_factory.mktemp("launches") / "norm_launches.so")
    subprocess.run([build.nvcc(), *build.ARCH, "-O1", "-std=c++17", "-Xcompiler", "-fPIC", "-shared", "-I", build.CSRC, "-I", build.INCLUDE,
                    os.path.join(HERE, "norm_launches.cu"), "-o", out], check=True)
    it = ctypes.CDLL(out)
    i64, i32 = ctypes.c_int64, ctypes.c_int32
    it.backward_of.argtypes = [i64, i64, i64, i64, i64, i32, i32, i32, ctypes.POINTER(Noted)]
    return it


def check(lib, rows, dim, samples, at=4096, pitch=None, flags=0, dw=1, db=1):
    """One call: every row is one CTA's, shifted as the CTA's others are, and every partial row has its place."""
    pitch = dim if pitch is None else pitch
    n = Noted()
    assert lib.backward_of(at, pitch, rows, dim, samples, flags, dw, db, ctypes.byref(n)) == abi.MXFP4_OK
    each, size = rows // samples, 4 if flags & abi.MXFP4_NORM_X_F32 else 2
    assert n.sample_rows == each and n.ctas == samples * n.chunks
    assert n.period in (1, 2, 4, 8) and (n.access == SHIFTED or n.period == 1)
    if n.access == SHIFTED:
        assert n.period * pitch * size % 16 == 0 or rows == 1
    # CTA c of a sample: rows c % period + (c / period) chunk_rows period, and every period-th behind it, chunk_rows of them at most
    seen = [0] * each
    for c in range(n.chunks):
        first = c % n.period + c // n.period * n.chunk_rows * n.period
        for r in range(first, min(first + n.chunk_rows * n.period, each), n.period):
            seen[r] += 1
    assert seen == [1] * each
    bytes_ = abi.mxfp4_layer_norm_workspace_bytes(dim)
    places = [(n.partial_w, dw, DW), (n.partial_b, db, DB)]
    if n.chunks == 1 or not (dw or db):   # dw and db themselves
        assert not n.reduced and all(p == (out if given else 0) for p, given, out in places)
        return n
    assert n.reduced == bool(dw) + bool(db) and (n.reduced_chunks, n.reduced_samples) == (n.chunks, samples)
    spans = sorted((p, p + 4 * n.ctas * dim) for p, given, _ in places if given)
    assert all((p != 0) == bool(given) for p, given, _ in places)
    assert spans[0][0] >= WORKSPACE and spans[-1][1] <= WORKSPACE + bytes_
    assert all(a[1] <= b[0] for a, b in zip(spans, spans[1:]))
    return n


@pytest.mark.parametrize("dim", [1, 77, 512, 513, 520, 1001, 1004, 1002, 4104, 4100, 8191, 16384])
def test_every_row_and_every_partial_row_has_its_place(lib, dim):
    kinds = set()
    for samples in list(range(1, 21)) + [37, 38, 39, 75, 76, 77, 151, 152, 153, 303, 304, 305, 306, 607, 608, 609, 700, 1215, 1217]:
        for each in (1, 2, 3, 4, 5, 7, 8, 9, 31, 33):
            n = check(lib, samples * each, dim, samples)
            kinds.add((n.access, n.period))
    for samples in (1, 2, 3, 19, 20, 37, 38, 39, 152, 153, 304, 305):
        for each in (303, 304, 1000, 1217, 4097):
            n = check(lib, samples * each, dim, samples)
            kinds.add((n.access, n.period))
    if dim > 512 and dim + 7 <= abi.MXFP4_NORM_MAX_DIM and dim % 8:   # rows of bf16 that start anywhere, and those that are too few for it
        period = {1: 8, 2: 4, 4: 2}[dim & -dim]
        assert kinds == {(0, 1), (SHIFTED, period)}
    else:
        assert all(period == 1 for _, period in kinds)


@pytest.mark.parametrize("samples", [1, 3, 19, 38, 39, 150])
@pytest.mark.parametrize("pitch, at", [(4104, 4096), (4105, 4098), (4106, 4098), (4108, 4102), (4112, 4110)])
def test_pitches_and_first_places(lib, samples, pitch, at):
    for each in (1, 6, 39, 200, 2000):
        check(lib, samples * each, 4100, samples, at, pitch)
        check(lib, samples * each, 4100, samples, at // 4 * 4, pitch, abi.MXFP4_NORM_X_F32)


@pytest.mark.parametrize("dw, db", [(0, 0), (1, 0), (0, 1)])
def test_one_gradient_or_none(lib, dw, db):
    for rows, dim, samples in ((5000, 1001, 1), (5000, 300, 2), (4, 300, 2), (4, 1001, 4)):
        check(lib, rows, dim, samples, dw=dw, db=db)
