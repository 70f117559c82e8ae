"""The launches of the gradients' norm over lists of every length, by the library's own host code, without a GPU."""
import ctypes
import os
import subprocess

import numpy as np
import pytest

from mxfp4_block_scaled_quantize_gb300 import abi, build

HERE = os.path.dirname(os.path.abspath(__file__))
MANY = 1280   # tensors of a launch
NOTED = np.dtype([(name, np.int64) for name in ("ctas", "tensors", "elements", "units", "slot", "slots")])


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    out = str(tmp_path_factory.mktemp("launches") / "grad_norm_launches.so")
    subprocess.run([build.nvcc(), *build.ARCH, "-O1", "-std=c++17", "-Xcompiler", "-fPIC", "-shared", "-I", build.CSRC, "-I", os.path.join(build.ROOT, "include"),
                    os.path.join(HERE, "grad_norm_launches.cu"), "-o", out], check=True)
    return ctypes.CDLL(out)


def launches(lib, sizes, flags):
    table = np.zeros(len(sizes), dtype=[("g", np.uint64), ("n", np.int64)])
    table["n"] = sizes
    table["g"] = 2 ** 20 + 16 * np.concatenate([[0], np.cumsum(np.array(sizes, dtype=np.int64) // 4 + 1)[:-1]]).astype(np.uint64)
    out, n = np.zeros(256, dtype=NOTED), ctypes.c_int64()
    status = lib.launches_of(len(sizes), ctypes.c_void_p(table.ctypes.data), flags, ctypes.c_void_p(out.ctypes.data), ctypes.byref(n))
    return status, out[:n.value]


@pytest.mark.parametrize("flags", range(4))
@pytest.mark.parametrize("sizes", [
    [5] * 1280, [5] * 1281, [5] * 1280 + [0], [5] * 1280 + [0] * 7, [0] * 3 + [5] * 1280 + [0], [5, 0] * 1280, [5] * 2560 + [0],
    [5] * 1280 + [0] + [5], [5] * 1280 + [0] * 2000 + [5] * 1280 + [0] * 2000, [5] * 48 + [0], [0, 5] * 30, [5] * 1279 + [2 ** 33] + [0],
    [2 ** 20] * 1300 + [0], [5] * 65535 + [0], [1] + [0] * 65535], ids=lambda s: f"{len(s)}_of_which_{sum(n > 0 for n in s)}")
def test_every_tensor_is_in_one_launch_and_every_slot_is_filled(lib, sizes, flags):
    status, found = launches(lib, sizes, flags)
    assert status == abi.MXFP4_OK
    full = sum(n > 0 for n in sizes)
    expected = -(-full // MANY) if len(sizes) > 48 else 1
    norm, scale = found[:expected], found[expected:]
    for part in (norm, scale) if flags & abi.MXFP4_GRAD_SCALE else (norm,):
        assert len(part) == expected and part["tensors"].sum() == full and part["elements"].sum() == sum(sizes)
        assert (part["ctas"] == np.minimum(part["units"], 4 * 152)).all() and (part["ctas"] > 0).all()
    assert len(scale) == (expected if flags & abi.MXFP4_GRAD_SCALE else 0)
    # the last CTA of all adds up the partial sums of all: side by side, none left out
    assert (norm["slots"] == norm["ctas"].sum()).all()
    assert (norm["slot"] == np.concatenate([[0], norm["ctas"].cumsum()[:-1]])).all()


@pytest.mark.parametrize("sizes", [[0], [0] * 49, [0] * 5000], ids=len)
def test_nothing_but_empty_tensors(lib, sizes):
    for flags in range(4):
        status, found = launches(lib, sizes, flags)
        assert status == abi.MXFP4_OK and len(found) == 1 and found["ctas"][0] == 1
