"""The MXFP4 linear of a mixture-of-experts layer: products grouped by expert, with group sizes
that only the device knows.

The routing gives, on the device, the rows of X for each expert: `rows` (int32 [R], the token of
every row of the grouped order, expert by expert) and `offsets` (int32 [E + 1], where each
expert's rows start).  The layer is `MXFP4Linear`'s data path per expert, in the same number of
launches whatever E is:

  forward    row (training: dual) quantization of the gathered rows of X and of W,
             Y_e = X_e . W_e^T                                            [R, N]
  backward   dual quantization of dY, dX_e = dY_e . W_e                   [R, K], grouped order
             and dW_e = dY_e^T . X_e                                      [E, N, K]

Nothing synchronizes with the host and nothing is allocated after construction, so a step can be
captured in a CUDA graph.  A server that holds its weights in MXFP4 calls `forward_packed`.
"""
import torch

from . import abi


def _addresses(blobs):
    return [b.data_ptr() for b in blobs] + [None] * (4 - len(blobs))


class MXFP4GroupedLinear:
    """groups experts with weights [N, K] and at most max_rows routed rows a call.  The results
    are views of the layer's own buffers and live until the next call."""

    def __init__(self, groups: int, N: int, K: int, max_rows: int, train: bool = True, device="cuda",
                 out_dtype=torch.bfloat16):
        if out_dtype not in (torch.bfloat16, torch.float32):
            raise ValueError(f"results in bf16 or fp32, not {out_dtype}")
        self.groups, self.N, self.K, self.max_rows, self.train = groups, N, K, max_rows, train
        code = abi.MXFP4_OUT_F32 if out_dtype == torch.float32 else abi.MXFP4_OUT_BF16
        self.x_blobs = abi.alloc_grouped_blobs(max_rows, K, groups, dual=train, device=device)
        self.y = torch.empty((max_rows, N), dtype=out_dtype, device=device)
        self._gpu = self._here(self.y)
        self._packed_bytes = abi.mxfp4_grouped_sizes(groups * N, K, groups, equal=True)[:2]
        self.w_blobs = None
        self._has_w = False   # w_blobs hold the blobs of some W
        self._away = False    # the products' weights are not w_blobs
        self._packed = False  # nor were they the last forward's
        self._rows = None     # its rows; None: no backward can follow
        self._c = abi.GroupedLinear(groups, N, K, out_dtype=code, y=self.y.data_ptr())
        self._c.x_blobs[:] = _addresses(self.x_blobs)
        if train:
            self._keep_w(abi.alloc_grouped_blobs(groups * N, K, groups, equal=True, device=device))
            self.dy_blobs = abi.alloc_grouped_blobs(max_rows, N, groups, device=device)
            self.dx = torch.empty((max_rows, K), dtype=out_dtype, device=device)
            self.dw = torch.empty((groups, N, K), dtype=out_dtype, device=device)
            self._c.dy_blobs[:] = _addresses(self.dy_blobs)
            self._c.dx, self._c.dw = self.dx.data_ptr(), self.dw.data_ptr()

    @staticmethod
    def _here(t):
        """Index of t's GPU; None elsewhere, which no tensor's get_device() is."""
        return t.get_device() if t.is_cuda else None

    # The checks are a call's host time next to its launch: few of torch's calls, no loops.
    @staticmethod
    def _elsewhere(what):
        return ValueError(f"{what}: the layer's tensors are on its GPU")

    def _check_rows(self, x, k, rows, offsets):
        """T, R and the pitch of x's rows."""
        shape = x.shape
        if x.dtype is not torch.bfloat16 or len(shape) != 2 or shape[1] != k or x.stride(1) != 1:
            raise ValueError(f"bf16 rows of {k} contiguous elements")
        gpu, T = self._gpu, shape[0]
        if rows is None:
            R = T
        else:
            R = rows.numel()
            if rows.dtype is not torch.int32 or not rows.is_contiguous():
                raise ValueError("rows: contiguous int32 values")
            if rows.get_device() != gpu:
                raise self._elsewhere("rows")
        if R > self.max_rows:
            raise ValueError(f"{R} rows for a layer of at most {self.max_rows}")
        if offsets.dtype is not torch.int32 or offsets.numel() != self.groups + 1 or not offsets.is_contiguous():
            raise ValueError(f"offsets: {self.groups + 1} contiguous int32 values")
        if x.get_device() != gpu or offsets.get_device() != gpu:
            raise self._elsewhere("rows and offsets")
        return T, R, abi.row_pitch(x)

    def _check_w(self, w):
        if w.dtype != torch.bfloat16 or w.shape != (self.groups, self.N, self.K) or not w.is_contiguous():
            raise ValueError(f"W: contiguous bf16 [{self.groups}, {self.N}, {self.K}]")
        if w.get_device() != self._gpu:
            raise self._elsewhere("W")
        if self.w_blobs is None:
            self._keep_w(abi.alloc_grouped_blobs(self.groups * self.N, self.K, self.groups, equal=True, dual=False,
                                                 device=w.device))

    def _keep_w(self, blobs):
        self.w_blobs = blobs
        self._c.w_blobs[:] = self._w_at = _addresses(blobs)

    def _check_packed(self, w_q, w_s):
        q, s = self._packed_bytes
        try:
            good = (w_q.element_size() == 1 and w_s.element_size() == 1 and w_q.numel() >= q and w_s.numel() >= s and
                    w_q.is_contiguous() and w_s.is_contiguous())
        except AttributeError:   # not tensors
            good = False
        if not good:
            raise ValueError(f"packed weights: contiguous bytes, {q} of codes and {s} of scales")
        if w_q.get_device() != self._gpu or w_s.get_device() != self._gpu:
            raise self._elsewhere("packed weights")

    def quantize_w(self, w, stream=None):
        """The blobs of W[E, N, K], kept for the products that follow (a forward and its backward use
        the same)."""
        self._check_w(w)
        blobs = self.w_blobs if self.train else self.w_blobs + (None, None)
        abi.mxfp4_quantize_grouped(w, self.groups * self.N, self.K, self.K, None, None, self.groups,
                                   self.groups * self.N, *blobs, stream)
        self._has_w, self._rows = True, None

    def _forward(self, x, w, offsets, rows, stream):
        T, R, ldx = self._check_rows(x, self.K, rows, offsets)
        abi.mxfp4_grouped_forward(self._c, x, T, ldx, rows, offsets, R, w, stream)
        self._rows = R
        return self.y if R == self.max_rows else self.y[:R]

    def forward(self, x, w, offsets, rows=None, stream=None):
        """Y [R, N] in the grouped order; w None: the weights of the last quantize_w or forward."""
        if w is not None:
            self._check_w(w)
        elif not self._has_w:
            raise ValueError("no weights quantized yet")
        if self._away:
            self._c.w_blobs[:], self._away = self._w_at, False
        y = self._forward(x, w, offsets, rows, stream)
        self._has_w, self._packed = True, False
        return y

    def forward_packed(self, x, w_q, w_s, offsets, rows=None, stream=None):
        """Y [R, N] with the row blob of the weights (codes [E * N, Kp / 2], scales in the tensor-core
        layout with each expert's rows padded to 128).  No backward follows it."""
        self._check_packed(w_q, w_s)
        self._away = True
        self._c.w_blobs[0], self._c.w_blobs[1] = w_q.data_ptr(), w_s.data_ptr()
        y = self._forward(x, None, offsets, rows, stream)
        self._packed = True
        return y

    def backward(self, dy, offsets, stream=None):
        """dX [R, K] in the grouped order (a token's rows are for the caller to add up) and
        dW [E, N, K], for the X, W and offsets of the last forward."""
        if not self.train:
            raise ValueError("backward needs the column blobs of a training layer")
        if self._packed:
            raise ValueError("the last forward took packed weights, which have no column blob")
        _, R, lddy = self._check_rows(dy, self.N, None, offsets)
        if R != self._rows:   # X's column blob is laid out for that forward's rows
            raise ValueError(f"{R} rows after " + ("no forward" if self._rows is None else
                                                   f"a forward of {self._rows} rows"))
        abi.mxfp4_grouped_backward(self._c, dy, lddy, offsets, R, stream)
        return self.dx if R == self.max_rows else self.dx[:R], self.dw

    def step(self, x, w, dy, offsets, rows=None, stream=None):
        y = self.forward(x, w, offsets, rows, stream)
        dx, dw = self.backward(dy, offsets, stream)
        return y, dx, dw
