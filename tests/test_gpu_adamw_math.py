"""The hand-written roots and quotients of AdamW's 8-bit moments against CUDA's rounded intrinsics."""
import ctypes
import os
import subprocess

import pytest
import torch

from mxfp4_block_scaled_quantize_gb300 import build

pytestmark = pytest.mark.gpu

HERE = os.path.dirname(os.path.abspath(__file__))


class Found(ctypes.Structure):
    _fields_ = [(name, ctypes.c_uint64) for name in ("checked", "bad", "worst", "where")]


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    # as the library is compiled
    out = str(tmp_path_factory.mktemp("math") / "adamw_math_check.so")
    subprocess.run([build.nvcc(), *build.ARCH, "-O3", "-std=c++17", "-Xcompiler", "-fPIC", "-shared", "-I", build.CSRC,
                    os.path.join(HERE, "adamw_math_check.cu"), "-o", out], check=True)
    torch.cuda.init()
    return ctypes.CDLL(out)


def found(call, *args):
    f = Found()
    assert call(ctypes.byref(f), *args) == 0
    return f


INF = 0x7F800000


# eight neighbours a call; eight values apart by a mantissa's half, a binade, and 2^28 floats (small and large in one call)
@pytest.mark.parametrize("stride", [1, 1 << 22, 1 << 23, 1 << 28])
def test_every_root(lib, stride):
    f = found(lib.check_roots, ctypes.c_uint32(INF), ctypes.c_uint32(stride))
    assert f.checked == INF + 1
    assert f.bad == 0, f"{f.bad} roots differ, one of bits {f.where:#x}"


# E4M3 spans quotients from 2^-10, below which all encodes to zero, to 448: xe = 10 .. -8
@pytest.mark.parametrize("se", [-89, -30, 0, 60, 118])
def test_quotients(lib, se):
    for xe in range(-8, 11):
        f = found(lib.check_quotients, se, xe, 16)
        assert f.checked >= 5 * 2 ** 23   # of 16 x 2^23, less those above 448 s in the largest binade
        assert f.bad == 0, f"{f.bad} quotients differ, one of s, x {f.where:#x}"


def test_quotients_at_the_end_of_the_range(lib):
    # x below 2^-100: 1.5 ulp before the correction, whose residual is wrong by no more than itself, and the last rounding
    for se in (-126, -120, -110, -100):
        for xe in range(-8, 11):
            f = found(lib.check_quotients, se, xe, 16)
            assert f.checked >= 5 * 2 ** 23 and f.worst <= 2
