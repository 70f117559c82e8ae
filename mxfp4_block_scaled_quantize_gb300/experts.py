"""A whole mixture-of-experts layer for a few tokens: routing, both products and the sum in one kernel.

What a decoding loop calls next to `MXFP4GroupedLinear`, which takes prompts and training steps.  From the router's
logits it chooses each token's experts, and gives

  y_t = sum_e w_e W2_e . (silu(g) * u),   [g; u] = W1_e . x_t

over weights that are held as MXFP4 row blobs (`abi.quantize_grouped(w, groups=experts, dual=False)`), an expert's rows of g
before its rows of u.  The activations are not quantized.  Nothing synchronizes with the host and nothing is allocated after
construction, so a step can be captured in a CUDA graph.
"""
import torch

from . import abi


class MXFP4Experts:
    """experts of W1 [2 inner, dim] and W2 [dim, inner], the top_k of them for each of at most max_tokens tokens.  normalize:
    the chosen experts' weights are divided by their sum, else they are the softmax over all experts.  The result is a
    view of the layer's own buffer and lives until the next call; calls of one layer, and replays of graphs that hold
    them, come one after the other."""

    def __init__(self, experts: int, dim: int, inner: int, top_k: int, max_tokens: int = abi.MXFP4_EXPERTS_MAX_TOKENS,
                 normalize: bool = True, device="cuda"):
        if not 1 <= max_tokens <= abi.MXFP4_EXPERTS_MAX_TOKENS:
            raise ValueError(f"1 to {abi.MXFP4_EXPERTS_MAX_TOKENS} tokens a call, not {max_tokens}: MXFP4GroupedLinear takes more")
        if not 1 <= top_k <= min(experts, abi.MXFP4_EXPERTS_MAX_TOP_K):
            raise ValueError(f"top_k from 1 to {min(experts, abi.MXFP4_EXPERTS_MAX_TOP_K)}, not {top_k}")
        self.experts, self.dim, self.inner, self.top_k = experts, dim, inner, top_k
        self.max_tokens, self.normalize = max_tokens, normalize
        size = abi.mxfp4_experts_workspace_bytes(max_tokens, experts, top_k, dim, inner)   # fewer tokens need less of everything
        self._workspace = torch.zeros(size, dtype=torch.uint8, device=device)
        self.y = torch.empty((max_tokens, dim), dtype=torch.bfloat16, device=device)
        self._gpu = self.y.get_device() if self.y.is_cuda else None   # no tensor's get_device() is None
        self._flags = abi.MXFP4_EXPERTS_NORMALIZE if normalize else 0
        self._bytes = (abi.mxfp4_grouped_sizes(experts * 2 * inner, dim, experts, equal=True)[:2] +
                       abi.mxfp4_grouped_sizes(experts * dim, inner, experts, equal=True)[:2])

    def _check_rows(self, v, n, what):
        if len(v.shape) != 2 or v.shape[1] != n or (n > 1 and v.stride(1) != 1):
            raise ValueError(f"{what}: rows of {n} contiguous elements")
        if v.get_device() != self._gpu:
            raise ValueError(f"{what}: the layer's tensors are on its GPU")
        if v.shape[0] > 1 and v.stride(0) < n:
            raise ValueError(f"{what}: rows that do not overlap")
        return v.shape[0], v.stride(0)

    def _check_packed(self, blobs):
        for b, n in zip(blobs, self._bytes):
            try:
                good = b.element_size() == 1 and b.numel() >= n and b.is_contiguous()
            except AttributeError:   # not a tensor
                good = False
            if not good:
                raise ValueError("packed weights: contiguous bytes, {} and {} of codes and scales of W1, {} and {} of W2"
                                 .format(*self._bytes))
            if b.get_device() != self._gpu:
                raise ValueError("packed weights: the layer's tensors are on its GPU")

    def forward(self, x, logits, up_q, up_s, down_q, down_s, stream=None):
        """Y [T, dim] in bf16 for bf16 x [T, dim] and logits [T, experts] in fp32 or bf16."""
        if x.dtype is not torch.bfloat16:
            raise ValueError(f"x: bf16, not {x.dtype}")
        if not abi.is_current(self._gpu):
            raise ValueError("the layer's GPU is not the current device")
        flags = self._flags
        if logits.dtype is torch.float32:
            flags |= abi.MXFP4_EXPERTS_LOGITS_F32
        elif logits.dtype is not torch.bfloat16:
            raise ValueError(f"logits: fp32 or bf16, not {logits.dtype}")
        tokens, ldx = self._check_rows(x, self.dim, "x")
        rows, ldl = self._check_rows(logits, self.experts, "logits")
        if rows != tokens or tokens > self.max_tokens:
            raise ValueError(f"{tokens} tokens and {rows} rows of logits for a layer of at most {self.max_tokens} tokens")
        self._check_packed((up_q, up_s, down_q, down_s))
        abi.mxfp4_experts_forward(x, tokens, ldx, logits, ldl, self.experts, self.top_k, self.dim, self.inner, up_q, up_s, down_q,
                                  down_s, self.y, self.dim, flags, self._workspace, self._workspace.numel(), stream)
        return self.y if tokens == self.max_tokens else self.y[:tokens]
