"""AdamW over the tensors of a model in one launch, with moments in fp32 or in 8 bits; the norm of all
gradients, and clipping by it.

The weight update next to the MXFP4 layers: it takes their dW (bf16 or fp32) and writes the bf16
W that the next step quantizes, from fp32 master copies where they are kept.
"""
import math
import operator

import numpy as np
import torch

from . import abi

_TABLE = np.dtype([(name, np.uint64) for name in ("p", "master", "g", "m", "v", "m_scale", "v_scale")] +
                  [("n", np.int64)])

_GRADS = np.dtype([("g", np.uint64), ("n", np.int64)])

_dtype = operator.attrgetter("dtype")
_elements, _contiguous = torch.Tensor.numel, torch.Tensor.is_contiguous
_device, _address = torch.Tensor.get_device, torch.Tensor.data_ptr


def _check_grads(grads, numel, gpu):
    """The type of the gradients, one for each count of numel, on GPU gpu."""
    dtype = grads[0].dtype
    if dtype not in (torch.float32, torch.bfloat16) or len(grads) != len(numel):
        raise ValueError("one fp32 or bf16 gradient for each parameter")
    # one of torch's functions after the other over all gradients, which takes less time than a loop's method calls
    if not (list(map(_dtype, grads)).count(dtype) == len(grads) and list(map(_elements, grads)) == numel and
            all(map(_contiguous, grads)) and list(map(_device, grads)).count(gpu) == len(grads)):
        raise ValueError("gradients: contiguous, of one type and the parameters' sizes, on the parameters' GPU")
    return dtype


class GradNorm:
    """The norm of all gradients of `params` (CUDA tensors: their sizes and GPU are taken).

    Its results are `out`, fp32 [norm, factor] on the GPU, factor = min(1, max_norm / (norm + 1e-6)); a NaN makes both NaN.
    They live until the next call, and calls of one GradNorm, or replays of graphs that hold them, come
    one after the other: give each of two that may overlap a GradNorm of its own."""

    def __init__(self, params):
        params = list(params)
        if not params:
            raise ValueError("no parameters")
        if len(params) > abi.MXFP4_GRAD_MAX_TENSORS:
            raise ValueError(f"{abi.MXFP4_GRAD_MAX_TENSORS} parameters at most")
        self._gpu = params[0].get_device() if params[0].is_cuda else None   # no tensor's get_device() is None
        self._numel = [p.numel() for p in params]
        self._table = np.zeros(len(params), dtype=_GRADS)
        self._table["n"] = self._numel
        self._find_table()
        self._workspace = torch.zeros(abi.mxfp4_grad_norm_workspace_bytes(len(params)), dtype=torch.uint8,
                                      device=params[0].device)
        self.out = torch.empty(2, dtype=torch.float32, device=params[0].device)

    def _find_table(self):
        self._grads = self._table["g"]   # a view and an address that every call uses
        self._address = self._table.ctypes.data

    def __setstate__(self, state):
        """A copy's table is its own."""
        self.__dict__.update(state)
        self._find_table()

    def measure(self, grads, max_norm=math.inf, stream=None):
        """`out` for these gradients (contiguous, all fp32 or all bf16, in the order of the parameters), which
        are only read: AdamW's step, given max_norm, does this and scales by the factor itself."""
        return self._run(list(map(_address, grads)), _check_grads(grads, self._numel, self._gpu), max_norm, 0, stream)

    def clip_(self, grads, max_norm, stream=None):
        """The same, and the gradients multiplied by the factor in place: no two share an element."""
        return self._run(list(map(_address, grads)), _check_grads(grads, self._numel, self._gpu), max_norm,
                         abi.MXFP4_GRAD_SCALE, stream)

    def _run(self, addresses, dtype, max_norm, flags, stream):
        if not max_norm > 0:
            raise ValueError(f"a largest norm above 0, not {max_norm}")
        if not abi.is_current(self._gpu):
            raise ValueError("the parameters' GPU is not the current device")
        self._grads[:] = addresses
        if dtype is torch.float32:
            flags |= abi.MXFP4_GRAD_F32
        abi.mxfp4_grad_norm(len(addresses), self._address, flags, max_norm, self.out, self._workspace,
                            self._workspace.numel(), stream)
        return self.out


class AdamW:
    """params: contiguous CUDA tensors, all fp32 or all bf16; masters: fp32 copies of bf16
    parameters (or None: the parameters themselves are updated).  Moments: `state_bits` 32 or 8
    allocates zeros; or exp_avg / exp_avg_sq give them, per tensor an fp32 tensor, or for 8 bits
    a pair (E4M3 codes, fp32 scale per 128 elements), exp_avg_sq then holding the square root of
    the second moment.  All tensors are updated in place and must stay where they are.

    seed: 8-bit moments are rounded stochastically, with random bits that seed, step and place
    decide, and follow their recurrences in expectation for every beta.  Without it they are
    rounded to nearest, and an element whose gradients shrink keeps its second moment for as long
    as a step moves it by less than half a code step relative to its block's largest; beta2 is
    then 0.95 at most, and 0.95 by default (else 0.999)."""

    def __init__(self, params, masters=None, state_bits=32, exp_avg=None, exp_avg_sq=None, lr=1e-3,
                 betas=None, eps=1e-8, weight_decay=0.01, seed=None):
        self.params = list(params)
        if not self.params:
            raise ValueError("no parameters")
        self.dtype = self.params[0].dtype
        if self.dtype not in (torch.float32, torch.bfloat16):
            raise ValueError(f"parameters in fp32 or bf16, not {self.dtype}")
        self.masters = None if masters is None else list(masters)
        if self.masters is not None and self.dtype == torch.float32:
            raise ValueError("fp32 parameters need no masters")
        if state_bits not in (8, 32):
            raise ValueError("state_bits: 32 or 8")
        if (exp_avg is None) != (exp_avg_sq is None):
            raise ValueError("exp_avg and exp_avg_sq: both, or neither")
        if exp_avg is None:
            exp_avg = [self._zeros(p, state_bits) for p in self.params]
            exp_avg_sq = [self._zeros(p, state_bits) for p in self.params]
        self.exp_avg, self.exp_avg_sq = list(exp_avg), list(exp_avg_sq)
        self.state_bits = 32 if isinstance(self.exp_avg[0], torch.Tensor) else 8
        if seed is not None and self.state_bits != 8:
            raise ValueError("seed: for 8-bit moments")
        to_nearest = self.state_bits == 8 and seed is None
        if betas is None:
            betas = (0.9, 0.95 if to_nearest else 0.999)
        elif to_nearest and betas[1] > 0.95:
            raise ValueError(f"8-bit moments rounded to nearest do not follow beta2 = {betas[1]}: give a seed, for "
                             "stochastic rounding, or beta2 up to 0.95")
        self.lr, self.betas, self.eps, self.weight_decay = lr, betas, eps, weight_decay
        self.seed = 0 if seed is None else seed & (2 ** 64 - 1)
        self._dynamic = 4 if seed is None else 5
        self._flags = (abi.MXFP4_ADAMW_P_F32 if self.dtype == torch.float32 else 0) | \
                      (abi.MXFP4_ADAMW_STATE_E4M3 if self.state_bits == 8 else 0) | \
                      (abi.MXFP4_ADAMW_STOCHASTIC if seed is not None else 0)
        self.steps = 0
        # made here, not at the first use: its workspace is zeroed once, which a step being captured would put off
        self.grad_norm = GradNorm(self.params) if len(self.params) <= abi.MXFP4_GRAD_MAX_TENSORS else None
        self._gpu = self.params[0].get_device() if self.params[0].is_cuda else None   # no tensor's get_device() is None
        self._numel = [p.numel() for p in self.params]
        self._table = np.zeros(len(self.params), dtype=_TABLE)
        self._find_table()
        self._fill()

    def _find_table(self):
        self._grads = self._table["g"]   # a view and an address that every step uses
        self._address = self._table.ctypes.data

    def __setstate__(self, state):
        """A copy's table is its own, and of its own tensors."""
        self.__dict__.update(state)
        self._find_table()
        self._fill()

    @staticmethod
    def _zeros(p, bits):
        if bits == 32:
            return torch.zeros(p.numel(), dtype=torch.float32, device=p.device)
        blocks = -(-p.numel() // abi.MXFP4_ADAMW_BLOCK)
        return (torch.zeros(p.numel(), dtype=torch.float8_e4m3fn, device=p.device),
                torch.zeros(blocks, dtype=torch.float32, device=p.device))

    def _fill(self):
        """Checks every tensor and writes the table that each step hands to the library."""
        def put(name, tensors, dtype, counts):
            if len(tensors) != len(self.params):
                raise ValueError(f"{len(tensors)} tensors of {name} for {len(self.params)} parameters")
            for t, n in zip(tensors, counts):
                if t.dtype != dtype or t.numel() != n or not t.is_contiguous() or t.device != self.params[0].device:
                    raise ValueError(f"{name}: contiguous {dtype} tensors of the parameters' sizes, on their device")
            self._table[name] = [t.data_ptr() for t in tensors]

        put("p", self.params, self.dtype, self._numel)
        if self.masters is not None:
            put("master", self.masters, torch.float32, self._numel)
        for name, moments in (("m", self.exp_avg), ("v", self.exp_avg_sq)):
            for x in moments:
                if isinstance(x, torch.Tensor) != (self.state_bits == 32) or (self.state_bits == 8 and len(x) != 2):
                    raise ValueError("moments: all fp32 tensors, or all pairs of E4M3 codes and scales")
            if self.state_bits == 32:
                put(name, moments, torch.float32, self._numel)
            else:
                put(name, [c for c, _ in moments], torch.float8_e4m3fn, self._numel)
                put(name + "_scale", [s for _, s in moments], torch.float32,
                    [-(-n // abi.MXFP4_ADAMW_BLOCK) for n in self._numel])
        self._table["n"] = self._numel

    def step(self, grads, step=None, lr=None, grad_scale=1.0, dynamic=None, stream=None, max_norm=None,
             grad_factor=None):
        """One update with the gradients (contiguous, all fp32 or all bf16, in the order of the
        parameters).  step: this step's number (default: counted from 1); grad_scale: a factor on
        every gradient; dynamic: a CUDA fp32 tensor [lr, 1 - beta1^step, 1 - beta2^step, grad_scale]
        (with a seed, and step) that takes their place, for steps captured in a graph.  max_norm: the
        gradients, as they are given, are scaled down to that norm where theirs is larger; their
        norm and the factor are then in `grad_norm.out`.  grad_factor: one CUDA fp32 that grad_scale is
        multiplied by, the factor of a GradNorm over more parameters than these (`out[1:]`)."""
        dtype = _check_grads(grads, self._numel, self._gpu)
        if dynamic is not None and (dynamic.dtype != torch.float32 or dynamic.numel() != self._dynamic or
                                    not dynamic.is_contiguous() or dynamic.get_device() != self._gpu):
            raise ValueError(f"dynamic: {self._dynamic} consecutive fp32 on the parameters' GPU")
        if grad_factor is not None and (max_norm is not None or grad_factor.dtype != torch.float32 or
                                        grad_factor.numel() != 1 or grad_factor.get_device() != self._gpu):
            raise ValueError("grad_factor: one fp32 on the parameters' GPU, and no max_norm beside it")
        if step is None:
            step = self.steps + 1
        addresses = list(map(_address, grads))
        self._grads[:] = addresses
        flags = self._flags | (abi.MXFP4_ADAMW_G_F32 if dtype == torch.float32 else 0)
        factor = None if grad_factor is None else grad_factor.data_ptr()
        if max_norm is not None:
            if self.grad_norm is None:
                raise ValueError(f"max_norm: for up to {abi.MXFP4_GRAD_MAX_TENSORS} parameters")
            self.grad_norm._run(addresses, dtype, max_norm, 0, stream)
            factor = self.grad_norm.out.data_ptr() + 4
        if factor is not None:
            flags |= abi.MXFP4_ADAMW_GRAD_FACTOR
        h = abi.AdamwParams(self.lr if lr is None else lr, self.betas[0], self.betas[1], self.eps, self.weight_decay,
                            grad_scale, step, None if dynamic is None else dynamic.data_ptr(), self.seed, factor)
        abi.mxfp4_adamw(len(self.params), self._address, flags, h, stream)
        self.steps = step
