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


class MXFP4GroupedLinear:
    """groups experts with weights [N, K] and at most max_rows routed rows a call.  The results
    are views of the layer's own buffers and live until the next call."""

    def __init__(self, groups: int, N: int, K: int, max_rows: int, train: bool = True, device="cuda",
                 out_dtype=torch.bfloat16):
        assert out_dtype in (torch.bfloat16, torch.float32)
        self.groups, self.N, self.K, self.max_rows, self.train = groups, N, K, max_rows, train
        self.code = abi.MXFP4_OUT_F32 if out_dtype == torch.float32 else abi.MXFP4_OUT_BF16
        self.x_blobs = abi.alloc_grouped_blobs(max_rows, K, groups, dual=train, device=device)
        self.y = torch.empty((max_rows, N), dtype=out_dtype, device=device)
        self.w_blobs = None
        if train:
            self.w_blobs = abi.alloc_grouped_blobs(groups * N, K, groups, equal=True, device=device)
            self.dy_blobs = abi.alloc_grouped_blobs(max_rows, N, groups, device=device)
            self.dx = torch.empty((max_rows, K), dtype=out_dtype, device=device)
            self.dw = torch.empty((groups, N, K), dtype=out_dtype, device=device)

    def _rows(self, x, offsets, rows) -> int:
        R = x.shape[0] if rows is None else rows.numel()
        if R > self.max_rows:
            raise ValueError(f"{R} rows for a layer of at most {self.max_rows}")
        if offsets.dtype != torch.int32 or offsets.numel() != self.groups + 1 or not offsets.is_contiguous():
            raise ValueError(f"offsets: {self.groups + 1} contiguous int32 values")
        if rows is not None and (rows.dtype != torch.int32 or not rows.is_contiguous()):
            raise ValueError("rows: contiguous int32 values")
        return R

    def _quantize(self, x, offsets, rows, R, k, blobs, stream):
        if x.dtype != torch.bfloat16 or x.dim() != 2 or x.shape[1] != k or x.stride(1) != 1:
            raise ValueError(f"bf16 rows of {k} contiguous elements")
        abi.mxfp4_quantize_grouped(x, x.shape[0], k, x.stride(0), rows, offsets, self.groups, R, *blobs, stream=stream)

    def quantize_w(self, w, stream=None):
        """The blobs of W[E, N, K], kept for the products of this step."""
        if w.dtype != torch.bfloat16 or tuple(w.shape) != (self.groups, self.N, self.K) or not w.is_contiguous():
            raise ValueError(f"W: contiguous bf16 [{self.groups}, {self.N}, {self.K}]")
        if self.w_blobs is None:
            self.w_blobs = abi.alloc_grouped_blobs(self.groups * self.N, self.K, self.groups, equal=True, dual=False,
                                                   device=w.device)
        self._quantize(w.view(-1, self.K), None, None, self.groups * self.N, self.K, self.w_blobs, stream)

    def forward(self, x, w, offsets, rows=None, stream=None):
        """Y [R, N] in the grouped order; w None: the weights of the last quantize_w."""
        if w is not None:
            self.quantize_w(w, stream)
        return self.forward_packed(x, self.w_blobs[0], self.w_blobs[1], offsets, rows, stream)

    def forward_packed(self, x, w_q, w_s, offsets, rows=None, stream=None):
        """Y [R, N] with the row blob of the weights (codes [E * N, Kp / 2], scales in the tensor-core
        layout with each expert's rows padded to 128)."""
        R = self._rows(x, offsets, rows)
        self._quantize(x, offsets, rows, R, self.K, self.x_blobs, stream)
        y = self.y[:R]
        abi.mxfp4_gemm_grouped(abi.MXFP4_GROUPED_FWD, *self.x_blobs[:2], w_q, w_s, offsets, self.groups, R, self.N,
                               self.K, y, self.N, self.code, stream)
        return y

    def backward(self, dy, offsets, stream=None):
        """dX [R, K] in the grouped order (a token's rows are for the caller to add up) and
        dW [E, N, K], for the X, W and offsets of the last forward."""
        assert self.train, "backward needs the column blobs of a training layer"
        R = self._rows(dy, offsets, None)
        self._quantize(dy, offsets, None, R, self.N, self.dy_blobs, stream)
        dx = self.dx[:R]
        abi.mxfp4_gemm_grouped(abi.MXFP4_GROUPED_DGRAD, *self.dy_blobs[:2], *self.w_blobs[2:], offsets, self.groups, R,
                               self.N, self.K, dx, self.K, self.code, stream)
        abi.mxfp4_gemm_grouped(abi.MXFP4_GROUPED_WGRAD, *self.dy_blobs[2:], *self.x_blobs[2:], offsets, self.groups, R,
                               self.N, self.K, self.dw, self.K, self.code, stream)
        return dx, self.dw

    def step(self, x, w, dy, offsets, rows=None, stream=None):
        y = self.forward(x, w, offsets, rows, stream)
        dx, dw = self.backward(dy, offsets, stream)
        return y, dx, dw
