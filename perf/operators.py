"""Workloads of the grouped MXFP4 linear and of the AdamW step, with their plain forms.

Three operators, each from one token or one small tensor up to a full training step:

  serve   Y_e = X_e . W_e^T for the experts of a mixture-of-experts layer: the rows of bf16 X
          that the routing sent to expert e are gathered, quantized to MXFP4 and multiplied by
          that expert's weights, which a server holds in MXFP4 (packed E2M1 codes, E8M0 scales
          in the tensor-core layout).  The groups are ragged and some are empty.
  train   the training step of such a layer: X, W and dY quantized along both of their axes,
          Y_e = X_e . W_e^T, dX_e = dY_e . W_e and dW_e = dY_e^T . X_e.
  adamw   one AdamW step over many tensors at once, with moments in 32 bits or in 8 (E4M3 codes
          with an fp32 scale per 128 elements; the second moment held as its square root).

`own` selects who computes: False, elementary torch operations; True, the library.
"""
import math

import torch

own = False

BLOCK = 32           # elements that share an MXFP4 scale
STATE_BLOCK = 128    # elements that share the scale of an 8-bit moment
E4M3_MAX = 448.0
F32_TINY = 2.0 ** -126

HYPER = {"lr": 1e-3, "beta1": 0.9, "beta2": 0.95, "eps": 1e-8, "weight_decay": 0.1, "step": 100}


# ---------------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------------
def listed():
    return [
        # one token of a decoding loop sent to 8 of 64 experts: the weights of 8 experts are read for 8 rows
        {"name": "serve_one_token", "op": "serve", "tokens": 1, "top_k": 8, "experts": 64, "n": 2048, "k": 2048, "f32": False},
        # a decoding batch of 32 sequences on 64 experts: a few rows each, nearly every expert used
        {"name": "serve_batch_32", "op": "serve", "tokens": 32, "top_k": 8, "experts": 64, "n": 2048, "k": 2048, "f32": False},
        # a short prompt with sizes off every tile edge, fp32 results (a last layer kept in fp32)
        {"name": "serve_odd_f32", "op": "serve", "tokens": 333, "top_k": 2, "experts": 7, "n": 1000, "k": 1544, "f32": True},
        # a long prompt (or several) through 32 experts of 4096 x 4096
        {"name": "serve_prompt_4096", "op": "serve", "tokens": 4096, "top_k": 4, "experts": 32, "n": 4096, "k": 4096, "f32": False},
        # a small model's step, where launches and ramp-up count
        {"name": "train_small", "op": "train", "tokens": 512, "top_k": 2, "experts": 8, "n": 512, "k": 512, "f32": False},
        # odd sizes in every direction, fp32 gradients for accumulation
        {"name": "train_odd_f32", "op": "train", "tokens": 1111, "top_k": 1, "experts": 5, "n": 1032, "k": 1416, "f32": True},
        # many narrow experts: few tokens for each, the weights and their gradients dominate
        {"name": "train_64_experts", "op": "train", "tokens": 4096, "top_k": 6, "experts": 64, "n": 1408, "k": 2048, "f32": False},
        # wide experts with many tokens each: the matrix products dominate
        {"name": "train_wide_8192", "op": "train", "tokens": 8192, "top_k": 2, "experts": 8, "n": 8192, "k": 2048, "f32": False},
        # the norms and biases of a small model: 24 tensors of a few thousand values, fp32 throughout
        {"name": "adamw_small_f32", "op": "adamw", "tensors": 24, "size": 3001, "param": "f32", "grad": "f32", "state": 32},
        # the weights of a model in bf16 with fp32 master copies and 32-bit moments
        {"name": "adamw_bf16_state32", "op": "adamw", "tensors": 48, "size": 1500000, "param": "bf16_master", "grad": "bf16", "state": 32},
        # the same with 8-bit moments, fp32 gradients (accumulated over micro-batches)
        {"name": "adamw_bf16_state8", "op": "adamw", "tensors": 200, "size": 700001, "param": "bf16_master", "grad": "f32", "state": 8},
        # the largest: 8-bit moments for a few hundred million weights
        {"name": "adamw_large_state8", "op": "adamw", "tensors": 32, "size": 9000000, "param": "bf16_master", "grad": "bf16", "state": 8},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["serve", "train", "adamw"])
    if op == "adamw":
        tensors = _log(rng, 1, 240)
        size = _log(rng, 500, min(8000000, 250000000 // tensors))
        return {"op": op, "tensors": tensors, "size": size, "param": rng.choice(["f32", "bf16_master", "bf16"]),
                "grad": rng.choice(["f32", "bf16"]), "state": rng.choice([32, 8])}
    experts = _log(rng, 2, 64)
    top_k = rng.randint(1, min(8, experts))
    side = 4096 if op == "serve" else 2048
    n = 8 * _log(rng, 16, side // 8)
    k = 8 * _log(rng, 16, side // 8)
    if rng.random() < 0.5:   # the usual widths are whole tiles
        n, k = max(128, n // 128 * 128), max(128, k // 128 * 128)
    most = 16384 // top_k if op == "serve" else 12288 // top_k
    tokens = _log(rng, 1, most) if op == "serve" else _log(rng, 64, most)
    return {"op": op, "tokens": tokens, "top_k": top_k, "experts": experts, "n": n, "k": k, "f32": rng.random() < 0.3}


def _pad(n, m=128):
    return (n + m - 1) // m * m


def work(case):
    if case["op"] == "adamw":
        count = sum(_sizes(case))
        p = {"f32": 4, "bf16": 2, "bf16_master": 6}[case["param"]]
        g = 4 if case["grad"] == "f32" else 2
        s = 8 if case["state"] == 32 else 2 + 8 / STATE_BLOCK
        # read: parameter (only the master where there is one), gradient, moments; write: parameter and master, moments
        read = (4 if case["param"] == "bf16_master" else p) + g + s
        return {"bytes": count * (read + p + s), "flops": 16 * count}
    t, e, n, k = case["tokens"], case["experts"], case["n"], case["k"]
    rows = t * case["top_k"]
    out = 4 if case["f32"] else 2
    if case["op"] == "serve":
        used = min(e, rows)
        return {"bytes": 2 * t * k + 4 * rows + used * n * (_pad(k) // 2 + _pad(k) // 32) + out * rows * n,
                "flops": 2 * rows * n * k}
    return {"bytes": 2 * (t * k + e * n * k + rows * n) + 4 * rows + out * (rows * n + rows * k + e * n * k),
            "flops": 6 * rows * n * k}


# ---------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------
def _route(tokens, top_k, experts, gen):
    """Routing of `tokens` tokens to `top_k` of `experts` experts with uneven popularity: the token of every row of the
    grouped order (int32), the groups' offsets (int32, experts + 1) and the rows of the largest group."""
    logits = torch.randn(tokens, experts, generator=gen, device="cuda")
    logits += 0.5 * torch.randn(experts, generator=gen, device="cuda")
    chosen = logits.topk(top_k, dim=1).indices.reshape(-1)
    order = torch.argsort(chosen, stable=True)
    counts = torch.bincount(chosen, minlength=experts)
    offsets = torch.zeros(experts + 1, dtype=torch.int32, device="cuda")
    offsets[1:] = counts.cumsum(0)
    return (order // top_k).to(torch.int32), offsets, int(counts.max())


def _activations(t, k, gen):
    x = torch.randn(t, k, generator=gen, device="cuda")
    x *= 1 + 15 * (torch.rand(k, generator=gen, device="cuda") < 0.01)   # a few channels with large values
    return x.to(torch.bfloat16)


def _pack(w):
    """bf16 W[E, N, K] as the blob that a server keeps: codes [E * N, Kp / 2] (element 2j in the low half of byte j) and
    the scale bytes of each expert's rows, padded to 128, in 128-row x 4-block atoms of 512 bytes."""
    e, n, k = w.shape
    kp, n_pad = _pad(k), _pad(n)
    v = torch.zeros(e, n, kp, device=w.device)
    v[:, :, :k] = w.float()
    v = v.view(e, n, kp // BLOCK, BLOCK)
    exp = (torch.frexp(v.abs().amax(-1))[1] - 3).clamp(-127, 127)
    exp = torch.where(v.abs().amax(-1) == 0, torch.full_like(exp, -127), exp)
    y = torch.ldexp(v, -exp.unsqueeze(-1))
    a = y.abs()
    # the code of a magnitude on {0, .5, 1, 1.5, 2, 3, 4, 6}, nearest, ties to the even code
    code = ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0))
    code = (code + 8 * torch.signbit(y)).to(torch.uint8).view(e * n, kp)
    q = code[:, 0::2] | (code[:, 1::2] << 4)
    s = torch.zeros(e, n_pad, kp // BLOCK, dtype=torch.uint8, device=w.device)
    s[:, :n] = (exp + 127).to(torch.uint8)
    s = s.view(e * n_pad // 128, 4, 32, kp // 128, 4).permute(0, 3, 2, 1, 4)
    return q.contiguous(), s.contiguous().view(-1)


def _sizes(case):
    """Element counts of the tensors: around `size`, from an eighth of it to twice as many."""
    n, size = case["tensors"], case["size"]
    return [max(1, int(size * (0.125 + 1.875 * ((i * 7919) % 101) / 100) / 1.0625)) for i in range(n)]


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    if case["op"] == "adamw":
        return _prepare_adamw(case, gen)
    t, n, k, e = case["tokens"], case["n"], case["k"], case["experts"]
    rows, offsets, most = _route(t, case["top_k"], e, gen)
    x = _activations(t, k, gen)
    w = (0.02 * torch.randn(e, n, k, generator=gen, device="cuda")).to(torch.bfloat16)
    state = {"op": case["op"], "x": x, "rows": rows, "offsets": offsets, "most": most, "n": n, "k": k, "experts": e,
             "dtype": torch.float32 if case["f32"] else torch.bfloat16}
    if case["op"] == "serve":
        state["w_q"], state["w_s"] = _pack(w)
    else:
        state["w"] = w
        state["dy"] = (1e-3 * torch.randn(rows.numel(), n, generator=gen, device="cuda")).to(torch.bfloat16)
    if own:   # the layer that a program keeps: buffers for its blobs and results
        from mxfp4_block_scaled_quantize_gb300.grouped import MXFP4GroupedLinear
        state["layer"] = MXFP4GroupedLinear(e, n, k, rows.numel(), train=case["op"] == "train", out_dtype=state["dtype"])
    return state


def _flat(counts, dtype, unit):
    """Zeroed storage for tensors of these counts, each starting at a multiple of `unit` elements, and their places."""
    at, places = 0, []
    for c in counts:
        places.append((at, c))
        at += _pad(c, unit)
    return torch.zeros(at, dtype=dtype, device="cuda"), places


def _views(flat, places):
    return [flat[a:a + c] for a, c in places]


def _prepare_adamw(case, gen):
    counts = _sizes(case)
    blocks = [(c + STATE_BLOCK - 1) // STATE_BLOCK for c in counts]

    def randn(flat, places, std):
        for v in _views(flat, places):
            v.copy_(std * torch.randn(v.numel(), generator=gen, device="cuda"))

    p, at = _flat(counts, torch.float32 if case["param"] == "f32" else torch.bfloat16, STATE_BLOCK)
    randn(p, at, 0.02)
    g = torch.zeros(p.numel(), dtype=torch.float32 if case["grad"] == "f32" else torch.bfloat16, device="cuda")
    randn(g, at, 1e-3)
    state = {"op": "adamw", "param": p, "grad": g, "at": at, "bits": case["state"], "master": None}
    if case["param"] == "bf16_master":
        state["master"] = p.float()
        state["master"] += 1e-5 * torch.randn(p.numel(), generator=gen, device="cuda") * (p != 0)
    if case["state"] == 32:
        state["m"], state["v"] = torch.zeros(p.numel(), device="cuda"), torch.zeros(p.numel(), device="cuda")
        randn(state["m"], at, 3e-4)
        randn(state["v"], at, 1e-3)
        state["v"] *= state["v"]
    else:
        state["m"], state["v"] = (torch.zeros(p.numel(), dtype=torch.float8_e4m3fn, device="cuda") for _ in range(2))
        state["m_scale"], state["scale_at"] = _flat(blocks, torch.float32, 1)
        state["v_scale"] = torch.zeros_like(state["m_scale"])
        for i, (a, c) in enumerate(at):
            s, b = state["scale_at"][i]
            m = 3e-4 * torch.randn(c, generator=gen, device="cuda")
            r = 1e-3 * torch.rand(c, generator=gen, device="cuda")
            state["m"][a:a + c], state["m_scale"][s:s + b] = _encode8(m)
            state["v"][a:a + c], state["v_scale"][s:s + b] = _encode8(r)
    if own:   # the optimizer that a program keeps: its tensors and the table it hands to the library
        from mxfp4_block_scaled_quantize_gb300.optim import AdamW
        masters = _views(state["master"], at) if state["master"] is not None else None
        moments = [(_views(state[a], at) if case["state"] == 32 else
                    list(zip(_views(state[a], at), _views(state[a + "_scale"], state["scale_at"])))) for a in ("m", "v")]
        state["optimizer"] = AdamW(_views(p, at), masters=masters, exp_avg=moments[0], exp_avg_sq=moments[1],
                                   lr=HYPER["lr"], betas=(HYPER["beta1"], HYPER["beta2"]), eps=HYPER["eps"],
                                   weight_decay=HYPER["weight_decay"])
        state["grads"] = _views(g, at)
    return state


# ---------------------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------------------
def run(state):
    return _run_own(state) if own else _run_plain(state)


def _run_own(s):
    if s["op"] == "serve":
        return s["layer"].forward_packed(s["x"], s["w_q"], s["w_s"], s["offsets"], s["rows"])
    if s["op"] == "train":
        return s["layer"].step(s["x"], s["w"], s["dy"], s["offsets"], s["rows"])
    s["optimizer"].step(s["grads"], step=HYPER["step"])
    return _adamw_outputs(s)


def _adamw_outputs(s):
    names = ["param", "master", "m", "v"] + (["m_scale", "v_scale"] if s["bits"] == 8 else [])
    return {n: s[n] for n in names if s[n] is not None}


def _run_plain(s):
    if s["op"] == "adamw":
        return _adamw_plain(s)
    # the groups side by side: row i is row place[i] of expert expert[i], padded to whole blocks
    rows, offsets = s["rows"].long(), s["offsets"].long()
    index = torch.arange(rows.numel(), device="cuda")
    expert = torch.searchsorted(offsets[1:].contiguous(), index, right=True)
    place = index - offsets[expert]
    most = _pad(s["most"], BLOCK)

    def grouped(t):
        out = torch.zeros(s["experts"], most, _pad(t.shape[1]), device="cuda")
        out[expert, place, :t.shape[1]] = t.float()
        return out

    x = grouped(s["x"][rows])
    if s["op"] == "serve":
        w = _unpack(s["w_q"], s["w_s"], s["experts"], s["n"])
        return torch.bmm(_mxfp4(x), w.transpose(1, 2))[expert, place].to(s["dtype"])
    n, k = s["n"], s["k"]
    w = torch.zeros(s["experts"], _pad(n), _pad(k), device="cuda")
    w[:, :n, :k] = s["w"].float()
    dy = grouped(s["dy"])
    y = torch.bmm(_mxfp4(x), _mxfp4(w).transpose(1, 2))[expert, place, :n]
    dx = torch.bmm(_mxfp4(dy), _mxfp4_t(w))[expert, place, :k]
    dw = torch.bmm(_mxfp4_t(dy).transpose(1, 2), _mxfp4_t(x))[:, :n, :k]
    return y.to(s["dtype"]), dx.to(s["dtype"]), dw.to(s["dtype"])


def _mxfp4(x):
    """The values that MXFP4 holds for fp32 x, blocks of 32 along the last axis: scale 2^(floor(log2 amax) - 2), elements
    to the nearest of {0, .5, 1, 1.5, 2, 3, 4, 6}, ties to even, saturating."""
    b = x.reshape(*x.shape[:-1], x.shape[-1] // BLOCK, BLOCK)
    e = torch.frexp(b.abs().amax(-1, keepdim=True))[1] - 3
    y = torch.ldexp(b, -e)
    step = torch.where(y.abs() < 2, 0.5, torch.where(y.abs() < 4, 1.0, 2.0))
    y = (torch.round(y / step) * step).clamp(-6, 6)
    return torch.ldexp(y, e).reshape(x.shape)


def _mxfp4_t(x):
    """The same with the blocks along the last axis but one."""
    return _mxfp4(x.transpose(-1, -2).contiguous()).transpose(-1, -2)


def _unpack(q, s, experts, n):
    values = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], device=q.device)
    values = torch.cat([values, -values])
    kp, n_pad = 2 * q.shape[1], _pad(n)
    code = torch.stack([q & 15, q >> 4], dim=-1).view(experts, n, kp // BLOCK, BLOCK)
    s = s.view(experts * n_pad // 128, kp // 128, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(experts, n_pad, kp // BLOCK)
    return torch.ldexp(values[code.int()], s[:, :n].int().unsqueeze(-1) - 127).view(experts, n, kp)


def _blocks(x):
    """x in blocks of STATE_BLOCK, the last one filled up with zeros."""
    b = torch.zeros(_pad(x.numel(), STATE_BLOCK), device=x.device, dtype=x.dtype)
    b[:x.numel()] = x
    return b.view(-1, STATE_BLOCK)


def _encode8(x, keep=False):
    """E4M3 codes of x and the fp32 scale of each block, amax / 448; with `keep` what is above zero stays above zero."""
    b = _blocks(x)
    scale = (b.abs().amax(1, keepdim=True) / E4M3_MAX).clamp(min=F32_TINY)
    y = b / scale
    if keep:
        y = torch.where(b > 0, y.clamp(min=2.0 ** -9), y)
    return y.clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn).view(-1)[:x.numel()], scale.view(-1)


def _decode8(codes, scale):
    return (_blocks(codes.float()) * scale.view(-1, 1)).view(-1)[:codes.numel()]


def _adamw_plain(s):
    h = HYPER
    c1, c2 = 1 - h["beta1"] ** h["step"], 1 - h["beta2"] ** h["step"]
    for i, (a, c) in enumerate(s["at"]):
        here = slice(a, a + c)
        p = s["param"][here] if s["master"] is None else s["master"][here]
        g, p = s["grad"][here].float(), p.float()
        if s["bits"] == 8:
            at, b = s["scale_at"][i]
            scales = slice(at, at + b)
            m = _decode8(s["m"][here], s["m_scale"][scales])
            v = _decode8(s["v"][here], s["v_scale"][scales]).square()
        else:
            m, v = s["m"][here], s["v"][here]
        m = h["beta1"] * m + (1 - h["beta1"]) * g
        v = h["beta2"] * v + (1 - h["beta2"]) * g * g
        p = p - h["lr"] * ((m / c1) / (torch.sqrt(v / c2) + h["eps"]) + h["weight_decay"] * p)
        if s["bits"] == 8:
            s["m"][here], s["m_scale"][scales] = _encode8(m)
            s["v"][here], s["v_scale"][scales] = _encode8(torch.sqrt(v), keep=True)
        else:
            s["m"][here], s["v"][here] = m, v
        if s["master"] is not None:
            s["master"][here] = p
        s["param"][here] = p
    return _adamw_outputs(s)


# ---------------------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------------------
def _grid64(x, axis):
    """MXFP4 values of x (64 bits) with blocks of 32 from the start of `axis`, counted rather than rounded: a magnitude's
    place on the grid is the number of midpoints below it (a midpoint itself goes to the even neighbour)."""
    x = x.movedim(axis, -1)
    n = x.shape[-1]
    b = torch.zeros(*x.shape[:-1], _pad(n, BLOCK), dtype=torch.float64, device=x.device)
    b[..., :n] = x
    b = b.unflatten(-1, (-1, BLOCK))
    top = b.abs().amax(-1, keepdim=True)
    scale = torch.exp2((torch.frexp(top)[1].double() - 3).clamp(-127, 127))
    a = (b / scale).abs()
    grid = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device=x.device)
    spot = torch.zeros_like(a, dtype=torch.int32)
    for i, mid in enumerate((0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0)):
        spot += (a >= mid) if i % 2 else (a > mid)
    y = (grid[spot] * scale).copysign(b)
    return y.flatten(-2)[..., :n].movedim(-1, axis)


def exact(case, seed):
    global own
    kept, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = kept
    if case["op"] == "adamw":
        return _exact_adamw(s)
    cut = s["offsets"].tolist()
    x = s["x"].double()[s["rows"].long()]
    if case["op"] == "serve":
        x = _grid64(x, 1)
        table = torch.tensor([0, 1, 2, 3, 4, 6, 8, 12], dtype=torch.float64, device="cuda") / 2
        y = torch.empty(x.shape[0], s["n"], dtype=torch.float64, device="cuda")
        kp, n_pad = 2 * s["w_q"].shape[1], _pad(s["n"])
        r, b = torch.arange(s["n"], device="cuda").unsqueeze(1), torch.arange(kp // BLOCK, device="cuda")
        for e in range(s["experts"]):
            if cut[e] == cut[e + 1]:
                continue
            q = s["w_q"][e * s["n"]:(e + 1) * s["n"]].int()
            code = torch.empty(s["n"], kp, dtype=torch.int32, device="cuda")
            code[:, 0::2], code[:, 1::2] = q % 16, q // 16
            w = table[code % 8] * (1 - 2 * (code // 8))
            row = e * n_pad + r   # the scale byte's place, from the layout's definition
            byte = s["w_s"][((row // 128) * (kp // 128) + b // 4) * 512 + (row % 32) * 16 + (row % 128) // 32 * 4 + b % 4]
            w = w * torch.exp2(byte.double() - 127).repeat_interleave(BLOCK, 1)
            y[cut[e]:cut[e + 1]] = x[cut[e]:cut[e + 1]] @ w[:, :s["k"]].T
        return y
    dy = s["dy"].double()
    y, dx = torch.empty_like(dy), torch.empty_like(x)
    dw = torch.zeros(s["experts"], s["n"], s["k"], dtype=torch.float64, device="cuda")
    for e in range(s["experts"]):
        at = slice(cut[e], cut[e + 1])
        if cut[e] == cut[e + 1]:
            continue
        w = s["w"][e].double()
        y[at] = _grid64(x[at], 1) @ _grid64(w, 1).T
        dx[at] = _grid64(dy[at], 1) @ _grid64(w, 0)
        dw[e] = _grid64(dy[at], 0).T @ _grid64(x[at], 0)
    return y, dx, dw


def _e4m3_64(x, floor):
    """x (64 bits, in units of the block's scale) on the E4M3 grid: 3 bits after the leading one, steps of 2^-9 below 2^-6."""
    a = x.abs()
    step = torch.exp2((torch.frexp(a)[1].double() - 1).clamp(min=-6) - 3)
    y = (torch.round(a / step) * step).clamp(max=E4M3_MAX)
    if floor:
        y = torch.where((a > 0) & (y == 0), torch.full_like(y, 2.0 ** -9), y)
    return y.copysign(x)


def _exact_adamw(s):
    h = HYPER
    out = {n: v.double() for n, v in _adamw_outputs(s).items()}
    for i, (a, c) in enumerate(s["at"]):
        here = slice(a, a + c)
        g = s["grad"][here].double()
        p = (s["param"] if s["master"] is None else s["master"])[here].double()
        m, v = out["m"][here].clone(), out["v"][here].clone()
        if s["bits"] == 8:
            at, b = s["scale_at"][i]
            block = torch.arange(c, device="cuda") // STATE_BLOCK
            m = m * out["m_scale"][at:at + b][block]
            v = (v * out["v_scale"][at:at + b][block]) ** 2
        m = m + (1 - h["beta1"]) * (g - m)
        v = v + (1 - h["beta2"]) * (g * g - v)
        change = m / (1 - h["beta1"] ** h["step"]) / (torch.sqrt(v / (1 - h["beta2"] ** h["step"])) + h["eps"])
        p = p - h["lr"] * (change + h["weight_decay"] * p)
        for name, value, floor in (("m", m, False), ("v", torch.sqrt(v), True)) if s["bits"] == 8 else ():
            top = torch.zeros(b, dtype=torch.float64, device="cuda").scatter_reduce(0, block, value.abs(), "amax")
            scale = (top / E4M3_MAX).clamp(min=F32_TINY)
            out[name][here] = _e4m3_64(value / scale[block], floor)
            out[name + "_scale"][at:at + b] = scale
        if s["bits"] == 32:
            out["m"][here], out["v"][here] = m, v
        out["param"][here] = p
        if s["master"] is not None:
            out["master"][here] = p
    return out
