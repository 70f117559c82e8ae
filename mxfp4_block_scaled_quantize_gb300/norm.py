"""Layer norm in front of the MXFP4 linears, with its backward pass.

  forward    y = (x - mu) r g + b for each row of X [R, dim], mu its mean, r = 1 / sqrt(var + eps)
  backward   dx, and the gradients dw and db of the vectors

weight and bias are [dim], or [samples, dim] for as many equal runs of consecutive rows (a batch whose
samples have a scale and a shift of their own); with add_one the gain g is 1 + weight, else weight.
Nothing synchronizes with the host and nothing is allocated after construction, so a step can be
captured in a CUDA graph.
"""
import torch

from . import abi


class LayerNorm:
    """Rows of `dim` elements in bf16 or fp32, at most max_rows a call, in at most max_samples samples.  The results
    are views of the layer's own buffers and live until the next call; the next call may have one as its rows, whose place its
    results then take (rows that overlap a result's in any other way are refused)."""

    def __init__(self, dim: int, max_rows: int, eps: float = 1e-5, dtype=torch.bfloat16, add_one: bool = False,
                 max_samples: int = 1, train: bool = True, device="cuda"):
        if dtype not in (torch.bfloat16, torch.float32):
            raise ValueError(f"rows in bf16 or fp32, not {dtype}")
        if not 1 <= dim <= abi.MXFP4_NORM_MAX_DIM:
            raise ValueError(f"rows of 1 to {abi.MXFP4_NORM_MAX_DIM} elements, not {dim}")
        if max_rows < 0 or max_samples < 1 or not eps >= 0:
            raise ValueError("max_rows from 0 on, max_samples from 1 on, eps from 0 on")
        self.dim, self.max_rows, self.eps, self.dtype = dim, max_rows, eps, dtype
        self.add_one, self.max_samples, self.train = add_one, max_samples, train
        self._flags = (abi.MXFP4_NORM_X_F32 if dtype == torch.float32 else 0) | (abi.MXFP4_NORM_ADD_ONE if add_one else 0)

        def buf(*shape, dtype=torch.float32):
            return torch.empty(shape, dtype=dtype, device=device)

        self.y = buf(max_rows, dim, dtype=dtype)
        self._gpu = self.y.get_device() if self.y.is_cuda else None   # no tensor's get_device() is None
        self.mean = self.rstd = None
        if train:
            self.dx = buf(max_rows, dim, dtype=dtype)
            self.mean, self.rstd = buf(max_rows), buf(max_rows)
            self.dw, self.db = buf(max_samples, dim), buf(max_samples, dim)
            self._workspace = buf(abi.mxfp4_layer_norm_workspace_bytes(dim), dtype=torch.uint8)
            self._vectors = {}   # views of dw and db by the shape of the vectors, each made once
        self._last = None   # rows, and shapes and type of the last forward's vectors; None: no backward can follow

    def __setstate__(self, state):
        """A copy's gradients are views of its own buffers."""
        self.__dict__.update(state)
        if self.train:
            self._vectors = {}

    def _check_rows(self, x, what):
        shape = x.shape
        if x.dtype is not self.dtype or len(shape) != 2 or shape[1] != self.dim or (x.stride(1) != 1 and self.dim > 1):
            raise ValueError(f"{what}: {self.dtype} rows of {self.dim} contiguous elements")
        if shape[0] > self.max_rows:
            raise ValueError(f"{shape[0]} rows for a layer of at most {self.max_rows}")
        if x.get_device() != self._gpu:
            raise ValueError(f"{what}: the layer's tensors are on its GPU")
        pitch = x.stride(0)
        if shape[0] > 1 and pitch < self.dim:
            raise ValueError(f"{what}: rows that do not overlap")
        return shape[0], pitch

    def _check_vector(self, v, rows, what):
        """The samples of v."""
        shape, dim = v.shape, self.dim
        samples = 1 if len(shape) == 1 else shape[0]
        if v.dtype not in (torch.bfloat16, torch.float32) or len(shape) not in (1, 2) or shape[-1] != dim or not v.is_contiguous():
            raise ValueError(f"{what}: contiguous bf16 or fp32 [{dim}] or [samples, {dim}]")
        if not 1 <= samples <= self.max_samples or rows % samples:
            raise ValueError(f"{what}: {samples} samples for {rows} rows and a layer of at most {self.max_samples}")
        if v.get_device() != self._gpu:
            raise ValueError(f"{what}: the layer's tensors are on its GPU")
        return samples

    def forward(self, x, weight=None, bias=None, stream=None):
        """Y [R, dim] in the type of the rows."""
        if not abi.is_current(self._gpu):
            raise ValueError("the layer's GPU is not the current device")
        rows, pitch = self._check_rows(x, "x")
        samples, flags, kind = 1, self._flags, None
        for v, what in ((weight, "weight"), (bias, "bias")):
            if v is None:
                continue
            samples = self._check_vector(v, rows, what)
            if kind is not None and kind != (v.dtype, v.shape):
                raise ValueError("weight and bias: of one type and shape")
            kind = (v.dtype, v.shape)
        if kind is not None and kind[0] is torch.float32:
            flags |= abi.MXFP4_NORM_W_F32
        abi.mxfp4_layer_norm(x, rows, self.dim, pitch, weight, bias, samples, self.eps, flags, self.y, self.dim, self.mean,
                             self.rstd, stream)
        self._last = (rows, samples, flags, kind, weight is not None, bias is not None)
        return self.y if rows == self.max_rows else self.y[:rows]

    def backward(self, dy, x, weight=None, stream=None):
        """dX [R, dim] in the type of the rows, dW and dB in fp32 and the shape of the vectors (None where the forward
        had none), for the X and weight of the last forward."""
        if not self.train:
            raise ValueError("backward needs the statistics of a training layer")
        if self._last is None:
            raise ValueError("no forward before")
        if not abi.is_current(self._gpu):
            raise ValueError("the layer's GPU is not the current device")
        rows, samples, flags, kind, has_weight, has_bias = self._last
        (n, pitch), (nx, ldx) = self._check_rows(dy, "dy"), self._check_rows(x, "x")
        if n != rows or nx != rows:
            raise ValueError(f"{n} rows of dy and {nx} of x after a forward of {rows}")
        if (weight is not None) != has_weight:
            raise ValueError("a weight where the forward had one")
        if weight is not None:
            self._check_vector(weight, rows, "weight")
            if (weight.dtype, weight.shape) != kind:
                raise ValueError("weight: of the forward's type and shape")
        dw, db = self.dw if has_weight else None, self.db if has_bias else None
        abi.mxfp4_layer_norm_backward(dy, pitch, x, rows, self.dim, ldx, weight, samples, flags, self.mean, self.rstd, self.dx,
                                      self.dim, dw, db, self._workspace, self._workspace.numel(), stream)

        if kind is not None and kind[1] not in self._vectors:
            self._vectors[kind[1]] = self.dw[:samples].view(kind[1]), self.db[:samples].view(kind[1])
        views = (None, None) if kind is None else self._vectors[kind[1]]
        return (self.dx if rows == self.max_rows else self.dx[:rows], views[0] if has_weight else None,
                views[1] if has_bias else None)
