"""GPU: after a wait for weights has run out, the few tokens' experts ask for no more of them, say so, and leave the GPU and their
workspace fit for the next call.  The kernel is the library's, with one barrier that expects an arrival more than there is."""
import ctypes
import os
import subprocess

import numpy as np
import pytest
import torch

from mxfp4_block_scaled_quantize_gb300 import abi, build
from mxfp4_block_scaled_quantize_gb300.experts import MXFP4Experts

pytestmark = pytest.mark.gpu

HERE = os.path.dirname(os.path.abspath(__file__))
TOKENS, EXPERTS, TOP_K, DIM, INNER = 16, 32, 8, 2048, 1408   # on 152 SMs every warp has more than 7 slices of W1, in any CTA
STAGES, WARPS = 4, 16


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    import __graft_entry__
    __graft_entry__.build()
    out = str(tmp_path_factory.mktemp("lost") / "experts_lost_copy.so")
    subprocess.run([build.nvcc(), *build.ARCH, "-O3", "-std=c++17", "-Xcompiler", "-fPIC", "-shared", "-I", build.CSRC, "-I", build.INCLUDE,
                    os.path.join(HERE, "experts_lost_copy.cu"), build.LIB, "-Xlinker", "-rpath," + os.path.dirname(build.LIB), "-o", out], check=True)
    torch.cuda.set_device(0)
    abi.load()
    it = ctypes.CDLL(out)
    it.mxfp4_experts_forward.argtypes = abi.load().mxfp4_experts_forward.argtypes
    assert abi.mxfp4_last_device_error() == abi.MXFP4_OK
    yield it
    assert abi.mxfp4_last_device_error() == abi.MXFP4_OK


class Problem:
    def __init__(self):
        g = torch.Generator(device="cuda").manual_seed(1)

        def rnd(*shape):
            return torch.randn(shape, generator=g, device="cuda").to(torch.bfloat16)

        self.x, self.logits = rnd(TOKENS, DIM), rnd(TOKENS, EXPERTS).float()
        self.up = abi.quantize_grouped(rnd(EXPERTS * 2 * INNER, DIM), groups=EXPERTS, dual=False)[:2]
        self.down = abi.quantize_grouped(rnd(EXPERTS * DIM, INNER), groups=EXPERTS, dual=False)[:2]
        self.layer = MXFP4Experts(EXPERTS, DIM, INNER, TOP_K, max_tokens=TOKENS)
        self.want = self.library().clone()

    def library(self):
        return self.layer.forward(self.x, self.logits, *self.up, *self.down)

    def checked(self, lib, cta, thread):
        """One call of the checked kernel: y, and the copies that each warp asked for."""
        assert lib.lose(cta, thread) == 0
        p = [t.data_ptr() for t in (*self.up, *self.down)]
        w = self.layer._workspace
        flags = abi.MXFP4_EXPERTS_NORMALIZE | abi.MXFP4_EXPERTS_LOGITS_F32
        status = lib.mxfp4_experts_forward(self.x.data_ptr(), TOKENS, DIM, self.logits.data_ptr(), EXPERTS, EXPERTS, TOP_K, DIM, INNER, *p,
                                           self.layer.y.data_ptr(), DIM, flags, w.data_ptr(), w.numel(), torch.cuda.current_stream().cuda_stream)
        assert status == abi.MXFP4_OK
        torch.cuda.synchronize()
        found = np.zeros((256, WARPS), dtype=np.int32)
        assert lib.counted(ctypes.c_void_p(found.ctypes.data)) == 0
        return self.layer.y, found


@pytest.fixture(scope="module")
def problem(lib):
    return Problem()


def test_without_a_loss(lib, problem):
    y, copies = problem.checked(lib, -1, -1)
    assert torch.equal(y, problem.want)
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    assert (copies[:sms] >= 2 * 8).all() and not copies[sms:].any()   # two copies a slice


@pytest.mark.parametrize("cta, warp", [(0, 0), (77, 5), (151, 15)])
@pytest.mark.parametrize("stage", range(STAGES))
def test_a_wait_that_runs_out(lib, problem, cta, warp, stage):
    _, before = problem.checked(lib, -1, -1)
    _, copies = problem.checked(lib, cta, warp * STAGES + stage)
    assert abi.mxfp4_last_device_error() == abi.MXFP4_ERR_TIMEOUT
    # slice number `stage` never came: the first STAGES, and one for each slice before it, and none of the second product
    assert copies[cta, warp] == 2 * (STAGES + stage)
    assert (copies[cta] <= before[cta]).all()
    others = np.arange(256) != cta
    assert (copies[others] == before[others]).all()
    # the next calls are as if nothing had been
    assert torch.equal(problem.library(), problem.want)
    assert torch.equal(problem.checked(lib, -1, -1)[0], problem.want)
    assert abi.mxfp4_last_device_error() == abi.MXFP4_OK
