"""AdamW over the tensors of a model in one launch, with moments in fp32 or in 8 bits.

The weight update next to the MXFP4 layers: it takes their dW (bf16 or fp32) and writes the bf16
W that the next step quantizes, from fp32 master copies where they are kept.
"""
import operator

import numpy as np
import torch

from . import abi

_TABLE = np.dtype([(name, np.uint64) for name in ("p", "master", "g", "m", "v", "m_scale", "v_scale")] +
                  [("n", np.int64)])

_dtype = operator.attrgetter("dtype")
_elements, _contiguous = torch.Tensor.numel, torch.Tensor.is_contiguous
_device, _address = torch.Tensor.get_device, torch.Tensor.data_ptr


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
        self._gpu = self.params[0].get_device() if self.params[0].is_cuda else None   # no tensor's get_device() is None
        self._numel = [p.numel() for p in self.params]
        self._table = np.zeros(len(self.params), dtype=_TABLE)
        self._grads = self._table["g"]   # a view and an address that every step uses
        self._address = self._table.ctypes.data
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

    def step(self, grads, step=None, lr=None, grad_scale=1.0, dynamic=None, stream=None):
        """One update with the gradients (contiguous, all fp32 or all bf16, in the order of the
        parameters).  step: this step's number (default: counted from 1); grad_scale: a factor on
        every gradient; dynamic: a CUDA fp32 tensor [lr, 1 - beta1^step, 1 - beta2^step, grad_scale]
        (with a seed, and step) that takes their place, for steps captured in a graph."""
        dtype = grads[0].dtype
        if dtype not in (torch.float32, torch.bfloat16) or len(grads) != len(self.params):
            raise ValueError("one fp32 or bf16 gradient for each parameter")
        # one of torch's functions after the other over all gradients, which takes less time than a loop's method calls
        if not (list(map(_dtype, grads)).count(dtype) == len(grads) and list(map(_elements, grads)) == self._numel and
                all(map(_contiguous, grads)) and list(map(_device, grads)).count(self._gpu) == len(grads)):
            raise ValueError("gradients: contiguous, of one type and the parameters' sizes, on the parameters' GPU")
        if dynamic is not None and (dynamic.dtype != torch.float32 or dynamic.numel() != self._dynamic or
                                    not dynamic.is_contiguous() or dynamic.get_device() != self._gpu):
            raise ValueError(f"dynamic: {self._dynamic} consecutive fp32 on the parameters' GPU")
        if step is None:
            step = self.steps + 1
        self._grads[:] = list(map(_address, grads))
        flags = self._flags | (abi.MXFP4_ADAMW_G_F32 if dtype == torch.float32 else 0)
        h = abi.AdamwParams(self.lr if lr is None else lr, self.betas[0], self.betas[1], self.eps, self.weight_decay,
                            grad_scale, step, None if dynamic is None else dynamic.data_ptr(), self.seed)
        abi.mxfp4_adamw(len(self.params), self._address, flags, h, stream)
        self.steps = step
