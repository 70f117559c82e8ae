"""Workloads of layer norm, of the gradients' norm and of a few tokens' experts, with their plain forms.

Three operators around the linears of a block, each from its smallest call to its largest:

  norm     layer norm of the rows of X, with no weight, with weight and bias, or with a weight (as 1 + w) and
           bias for each sample of the batch (modulation); alone, or with its backward pass: dX, dW and db.
  clip     the norm of all gradients of a model, alone or with the gradients scaled down to a largest norm.
  experts  a whole mixture-of-experts layer for a few tokens: softmax of the router's logits, the top_k
           experts, Y_t = sum_j w_j . W2_j . (silu(G) * U) with [G; U] = W1_j . X_t, over weights that a
           server holds in MXFP4 (packed E2M1 codes, E8M0 scales in the tensor-core layout).

`own` selects who computes: False, elementary torch operations; True, the library.
"""
import math

import torch

own = False

BLOCK = 32           # elements that share an MXFP4 scale
EPS = 1e-5           # of the norm's variance
CLIP_EPS = 1e-6      # added to the gradients' norm before the division
MAX_NORM = 1.0
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---------------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------------
def listed():
    return [
        # one token of a decoding loop: latency alone
        {"name": "norm_one_token", "op": "norm", "rows": 1, "dim": 4096, "dtype": "bf16", "affine": "bf16", "samples": 1, "train": False},
        # a long prompt through the norm in front of a layer
        {"name": "norm_prompt", "op": "norm", "rows": 8192, "dim": 4096, "dtype": "bf16", "affine": "f32", "samples": 1, "train": False},
        # a training step of odd sizes kept in fp32
        {"name": "norm_train_odd_f32", "op": "norm", "rows": 1111, "dim": 1001, "dtype": "f32", "affine": "f32", "samples": 1, "train": True},
        # a training step with modulation: two samples, each with its own scale and shift
        {"name": "norm_train_modulated", "op": "norm", "rows": 4608, "dim": 5120, "dtype": "bf16", "affine": "bf16", "samples": 2, "train": True},
        # a training step of a wide model, the largest
        {"name": "norm_train_wide", "op": "norm", "rows": 16384, "dim": 8192, "dtype": "bf16", "affine": "f32", "samples": 1, "train": True},
        # the gradients of a small model, clipped: launches and the host's part count
        {"name": "clip_small_f32", "op": "clip", "tensors": 24, "size": 3001, "grad": "f32", "scale": True},
        # the norm of many gradients of odd sizes, for the optimizer to scale by
        {"name": "clip_norm_bf16", "op": "clip", "tensors": 200, "size": 700001, "grad": "bf16", "scale": False},
        # a few hundred million gradients, clipped in place
        {"name": "clip_large_bf16", "op": "clip", "tensors": 32, "size": 9000000, "grad": "bf16", "scale": True},
        # one token of a decoding loop sent to 8 of 64 experts
        {"name": "experts_one_token", "op": "experts", "tokens": 1, "top_k": 8, "experts": 64, "dim": 2048, "inner": 1408, "logits": "f32", "masked": False},
        # a decoding batch of 32 sequences on the same layer
        {"name": "experts_batch_32", "op": "experts", "tokens": 32, "top_k": 8, "experts": 64, "dim": 2048, "inner": 1408, "logits": "f32", "masked": False},
        # sizes off every tile edge, bf16 logits with ties, an expert switched off, a batch padded with empty rows
        {"name": "experts_odd_masked", "op": "experts", "tokens": 13, "top_k": 2, "experts": 7, "dim": 1000, "inner": 712, "logits": "bf16", "masked": True},
        # the largest batch that counts as few tokens, on wide experts
        {"name": "experts_batch_64", "op": "experts", "tokens": 64, "top_k": 6, "experts": 64, "dim": 4096, "inner": 2048, "logits": "f32", "masked": False},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "clip", "experts"])
    if op == "norm":
        dim = _log(rng, 64, 8192)
        if rng.random() < 0.5:   # the usual widths
            dim = max(128, dim // 128 * 128)
        samples = rng.choice([1, 1, 2, 3])
        rows = samples * _log(rng, 1, 16384 // samples)
        return {"op": op, "rows": rows, "dim": dim, "dtype": rng.choice(["bf16", "f32"]) if rows * dim <= 2 ** 25 else "bf16",
                "affine": rng.choice(["none", "bf16", "f32"]) if samples == 1 else rng.choice(["bf16", "f32"]),
                "samples": samples, "train": rng.random() < 0.6}
    if op == "clip":
        tensors = _log(rng, 1, 240)
        grad = rng.choice(["f32", "bf16"])
        return {"op": op, "tensors": tensors, "size": _log(rng, 500, min(8000000, (120000000 if grad == "f32" else 250000000) // tensors)),
                "grad": grad, "scale": rng.random() < 0.5}
    experts = _log(rng, 2, 64)
    dim, inner = _log(rng, 128, 4096), _log(rng, 128, 2048)
    if rng.random() < 0.6:
        dim, inner = max(128, dim // 128 * 128), max(128, inner // 64 * 64)
    masked = experts > 3 and rng.random() < 0.3
    return {"op": op, "tokens": _log(rng, 1, 64), "top_k": rng.randint(1, min(6, experts - masked)), "experts": experts, "dim": dim,
            "inner": inner, "logits": rng.choice(["f32", "bf16"]), "masked": masked}


def _pad(n, m=128):
    return (n + m - 1) // m * m


def work(case):
    if case["op"] == "norm":
        n, e = case["rows"] * case["dim"], 4 if case["dtype"] == "f32" else 2
        vectors = 0 if case["affine"] == "none" else 2 * case["samples"] * case["dim"]
        ve = 4 if case["affine"] == "f32" else 2
        if not case["train"]:
            return {"bytes": 2 * n * e + vectors * ve, "flops": 8 * n}
        # x, dy in; y, dx out; the vectors and their gradients
        return {"bytes": 4 * n * e + vectors * (ve + 4), "flops": 20 * n}
    if case["op"] == "clip":
        n, e = sum(_sizes(case)), 4 if case["grad"] == "f32" else 2
        return {"bytes": n * e * (2 if case["scale"] else 1), "flops": n * (3 if case["scale"] else 2)}
    t, e, k, d, i = case["tokens"], case["experts"], case["top_k"], case["dim"], case["inner"]
    used = e * (1 - (1 - k / e) ** t)   # experts that t tokens reach when all are alike
    weights = 2 * i * (_pad(d) // 2 + _pad(d) // 32) + d * (_pad(i) // 2 + _pad(i) // 32)
    return {"bytes": int(used * weights) + 4 * t * d + t * e * (4 if case["logits"] == "f32" else 2), "flops": 6 * t * k * d * i}


# ---------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------
def _activations(t, k, gen):
    x = torch.randn(t, k, generator=gen, device="cuda")
    x *= 1 + 15 * (torch.rand(k, generator=gen, device="cuda") < 0.01)   # a few channels with large values
    return x


def _pack(w):
    """fp32 W[N, K] as the blob that a server keeps: codes [N, Kp / 2] (element 2j in the low half of byte j) and the scale
    bytes, rows padded to 128, in 128-row x 4-block atoms of 512 bytes."""
    n, k = w.shape
    kp, n_pad = _pad(k), _pad(n)
    v = torch.zeros(n, kp, device=w.device)
    v[:, :k] = w
    v = v.view(n, kp // BLOCK, BLOCK)
    top = v.abs().amax(-1)
    exp = torch.where(top == 0, -127, (torch.frexp(top)[1] - 3).clamp(-127, 127))
    y = torch.ldexp(v, -exp.unsqueeze(-1))
    a = y.abs()
    # the code of a magnitude on {0, .5, 1, 1.5, 2, 3, 4, 6}, nearest, ties to the even code
    code = ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0))
    code = (code + 8 * torch.signbit(y)).to(torch.uint8).view(n, kp)
    s = torch.zeros(n_pad, kp // BLOCK, dtype=torch.uint8, device=w.device)
    s[:n] = (exp + 127).to(torch.uint8)
    s = s.view(n_pad // 128, 4, 32, kp // 128, 4).permute(0, 3, 2, 1, 4)
    return code[:, 0::2] | (code[:, 1::2] << 4), s.reshape(-1)


def _packed(experts, n, k, gen):
    """Codes [E * N, Kp / 2] and scale bytes of E experts' random weights."""
    q = torch.empty(experts * n, _pad(k) // 2, dtype=torch.uint8, device="cuda")
    s = torch.empty(experts, _pad(n) * (_pad(k) // BLOCK), dtype=torch.uint8, device="cuda")
    for e in range(experts):
        q[e * n:(e + 1) * n], s[e] = _pack(0.02 * torch.randn(n, k, generator=gen, device="cuda"))
    return q, s.view(-1)


def _sizes(case):
    """Element counts of the tensors: around `size`, from an eighth of it to twice as many."""
    n, size = case["tensors"], case["size"]
    return [max(1, int(size * (0.125 + 1.875 * ((i * 7919) % 101) / 100) / 1.0625)) for i in range(n)]


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    return {"norm": _prepare_norm, "clip": _prepare_clip, "experts": _prepare_experts}[case["op"]](case, gen)


def _prepare_norm(case, gen):
    r, d, dtype = case["rows"], case["dim"], TYPES[case["dtype"]]
    x = _activations(r, d, gen)
    x += 0.5 * torch.randn(r, 1, generator=gen, device="cuda")
    state = {"op": "norm", "x": x.to(dtype), "weight": None, "bias": None, "samples": case["samples"], "train": case["train"],
             "modulated": case["samples"] > 1}
    if case["affine"] != "none":
        shape = (case["samples"], d) if case["samples"] > 1 else (d,)
        centre = 0.0 if case["samples"] > 1 else 1.0   # modulation keeps the weight's distance from one
        state["weight"] = (centre + 0.2 * torch.randn(shape, generator=gen, device="cuda")).to(TYPES[case["affine"]])
        state["bias"] = (0.2 * torch.randn(shape, generator=gen, device="cuda")).to(TYPES[case["affine"]])
    if case["train"]:
        state["dy"] = (1e-3 * torch.randn(r, d, generator=gen, device="cuda")).to(dtype)
    if own:   # the layer that a program keeps: its results, statistics and workspace
        from mxfp4_block_scaled_quantize_gb300.norm import LayerNorm
        state["layer"] = LayerNorm(d, r, eps=EPS, dtype=dtype, add_one=state["modulated"], max_samples=case["samples"], train=case["train"])
    return state


def _prepare_clip(case, gen):
    counts = _sizes(case)
    flat = torch.zeros(sum(_pad(c) for c in counts), dtype=TYPES[case["grad"]], device="cuda")
    grads, at = [], 0
    for c in counts:
        grads.append(flat[at:at + c])
        grads[-1].copy_(1e-3 * torch.randn(c, generator=gen, device="cuda"))
        at += _pad(c)
    grads[-1].mul_(3.0 / grads[-1].float().norm())   # above the largest norm for every size
    state = {"op": "clip", "flat": flat, "grads": grads, "scale": case["scale"]}
    if own:   # the table and workspace that a program keeps for its parameters
        from mxfp4_block_scaled_quantize_gb300.optim import GradNorm
        state["norm"] = GradNorm(grads)
    return state


def _prepare_experts(case, gen):
    t, e, d, i = case["tokens"], case["experts"], case["dim"], case["inner"]
    state = {"op": "experts", "top_k": case["top_k"], "experts": e, "dim": d, "inner": i}
    state["x"] = _activations(t, d, gen).to(torch.bfloat16)
    logits = 1.5 * torch.randn(t, e, generator=gen, device="cuda") + 0.5 * torch.randn(e, generator=gen, device="cuda")
    logits = logits.to(TYPES[case["logits"]])
    if case["masked"]:
        logits[:, e // 2] = torch.finfo(logits.dtype).min   # an expert that takes nothing
        logits[t - t // 4:] = -math.inf                     # rows that pad the batch
    state["logits"] = logits
    state["up"] = _packed(e, 2 * i, d, gen)
    state["down"] = _packed(e, d, i, gen)
    if own:   # the layer that a program keeps: its results and workspace
        from mxfp4_block_scaled_quantize_gb300.experts import MXFP4Experts
        state["layer"] = MXFP4Experts(e, d, i, case["top_k"], max_tokens=t)
    return state


# ---------------------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------------------
def run(state):
    return _run_own(state) if own else _run_plain(state)


def _run_own(s):
    if s["op"] == "norm":
        y = s["layer"].forward(s["x"], s["weight"], s["bias"])
        if not s["train"]:
            return y
        return (y,) + tuple(g for g in s["layer"].backward(s["dy"], s["x"], s["weight"]) if g is not None)
    if s["op"] == "clip":
        if s["scale"]:
            return s["norm"].clip_(s["grads"], MAX_NORM), s["flat"]
        return s["norm"].measure(s["grads"], MAX_NORM)
    return s["layer"].forward(s["x"], s["logits"], *s["up"], *s["down"])


def _run_plain(s):
    return {"norm": _norm_plain, "clip": _clip_plain, "experts": _experts_plain}[s["op"]](s)


def _rows_of(v, rows):
    """The vectors [D] or [S, D], one for each of `rows` rows."""
    return v if v.dim() == 1 else v.repeat_interleave(rows // v.shape[0], 0)


def _norm_plain(s):
    x = s["x"].float()
    centred = x - x.mean(1, keepdim=True)
    rstd = 1 / torch.sqrt((centred * centred).mean(1, keepdim=True) + EPS)
    xh = centred * rstd
    gain = None
    y = xh
    if s["weight"] is not None:
        gain = _rows_of(s["weight"].float() + (1.0 if s["modulated"] else 0.0), x.shape[0])
        y = xh * gain + _rows_of(s["bias"].float(), x.shape[0])
    y = y.to(s["x"].dtype)
    if not s["train"]:
        return y
    dy = s["dy"].float()
    a = dy if gain is None else dy * gain
    dx = (rstd * (a - a.mean(1, keepdim=True) - xh * (a * xh).mean(1, keepdim=True))).to(s["x"].dtype)
    if gain is None:
        return y, dx
    shape = (s["samples"], -1, x.shape[1])
    dw, db = (dy * xh).view(shape).sum(1), dy.view(shape).sum(1)
    return y, dx, dw.view(s["weight"].shape), db.view(s["weight"].shape)


def _clip_plain(s):
    total = sum(g.float().square().sum(dtype=torch.float64) for g in s["grads"])
    norm = torch.sqrt(total)
    factor = (MAX_NORM / (norm + CLIP_EPS)).clamp(max=1.0).float()
    if not s["scale"]:
        return torch.stack([norm.float(), factor])
    for g in s["grads"]:
        g.copy_(g.float() * factor)
    return torch.stack([norm.float(), factor]), s["flat"]


def _gates(logits, top_k):
    """Weights [T, E] of the experts, zero where one is not chosen."""
    chosen = torch.sort(logits, dim=1, descending=True, stable=True).indices[:, :top_k]
    p = torch.exp(logits - logits.amax(1, keepdim=True))
    p = torch.where(torch.isneginf(logits), torch.zeros_like(p), p)
    p = p.gather(1, chosen)
    total = p.sum(1, keepdim=True)
    p = torch.where(total == 0, torch.zeros_like(p), p / total)
    return torch.zeros_like(logits).scatter(1, chosen, p)


def _unpack(q, s, expert, n):
    values = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], device=q.device)
    values = torch.cat([values, -values])
    kp, n_pad = 2 * q.shape[1], _pad(n)
    q = q[expert * n:(expert + 1) * n]
    s = s.view(-1, n_pad * kp // BLOCK)[expert]
    code = torch.stack([q & 15, q >> 4], dim=-1).view(n, kp // BLOCK, BLOCK)
    s = s.view(n_pad // 128, kp // 128, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(n_pad, kp // BLOCK)
    return torch.ldexp(values[code.int()], s[:n].int().unsqueeze(-1) - 127).view(n, kp)


def _experts_plain(s):
    x, d, i = s["x"].float(), s["dim"], s["inner"]
    gates = _gates(s["logits"].float(), s["top_k"])
    y = torch.zeros_like(x)
    for e in range(s["experts"]):
        h = x @ _unpack(*s["up"], e, 2 * i)[:, :d].T
        g, u = h[:, :i], h[:, i:]
        out = (g / (1 + torch.exp(-g)) * u) @ _unpack(*s["down"], e, d)[:, :i].T
        w = gates[:, e:e + 1]
        y += torch.where(w == 0, torch.zeros_like(out), w * out)
    return y.to(torch.bfloat16)


# ---------------------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------------------
def exact(case, seed):
    global own
    kept, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = kept
    return {"norm": _exact_norm, "clip": _exact_clip, "experts": _exact_experts}[case["op"]](s)


def _exact_norm(s):
    x = s["x"].double()
    r, d = x.shape
    mu = x.sum(1) / d
    xh = (x - mu[:, None]) / torch.sqrt(((x - mu[:, None]) ** 2).sum(1) / d + EPS)[:, None]
    rs = torch.sqrt(((x - mu[:, None]) ** 2).sum(1) / d + EPS)
    y = xh.clone()
    groups = [slice(k * (r // s["samples"]), (k + 1) * (r // s["samples"])) for k in range(s["samples"])]
    if s["weight"] is not None:
        w, b = s["weight"].double().view(s["samples"], d), s["bias"].double().view(s["samples"], d)
        if s["modulated"]:
            w = w + 1
        for k, at in enumerate(groups):
            y[at] = xh[at] * w[k] + b[k]
    if not s["train"]:
        return y
    dy = s["dy"].double()
    a = dy.clone()
    if s["weight"] is not None:
        for k, at in enumerate(groups):
            a[at] = dy[at] * w[k]
    dx = (a - (a.sum(1) / d)[:, None] - xh * ((a * xh).sum(1) / d)[:, None]) / rs[:, None]
    if s["weight"] is None:
        return y, dx
    dw = torch.stack([torch.einsum("rd,rd->d", dy[at], xh[at]) for at in groups])
    db = torch.stack([dy[at].sum(0) for at in groups])
    return y, dx, dw.view(s["weight"].shape), db.view(s["weight"].shape)


def _exact_clip(s):
    total = torch.zeros((), dtype=torch.float64, device="cuda")
    for g in s["grads"]:
        for piece in g.split(1 << 24):
            v = piece.double()
            total += torch.dot(v, v)
    norm = total.sqrt()
    factor = torch.minimum(torch.ones_like(norm), MAX_NORM / (norm + CLIP_EPS))
    pair = torch.stack([norm, factor])
    return (pair, s["flat"].double() * factor) if s["scale"] else pair


def _exact_experts(s):
    x, logits = s["x"].double(), s["logits"].double().cpu().tolist()
    d, i = s["dim"], s["inner"]
    y = torch.zeros_like(x)
    routed = {}
    for t, row in enumerate(logits):
        best = sorted(range(len(row)), key=lambda j: (-row[j], j))[:s["top_k"]]
        top = row[best[0]]
        if top == -math.inf:
            continue
        p = [math.exp(row[j] - top) for j in best]
        for j, w in zip(best, p):
            if w > 0:
                routed.setdefault(j, []).append((t, w / sum(p)))
    table = torch.tensor([0, 1, 2, 3, 4, 6, 8, 12], dtype=torch.float64, device="cuda") / 2

    def weights(blob, e, n, k):
        q, scale = blob
        kp, n_pad = 2 * q.shape[1], _pad(n)
        q = q[e * n:(e + 1) * n].int()
        code = torch.empty(n, kp, dtype=torch.int32, device="cuda")
        code[:, 0::2], code[:, 1::2] = q % 16, q // 16
        row = e * n_pad + torch.arange(n, device="cuda").unsqueeze(1)
        b = torch.arange(kp // BLOCK, device="cuda")
        # the scale byte's place, from the layout's definition
        byte = scale[((row // 128) * (kp // 128) + b // 4) * 512 + (row % 32) * 16 + (row % 128) // 32 * 4 + b % 4]
        w = table[code % 8] * (1 - 2 * (code // 8)) * torch.exp2(byte.double() - 127).repeat_interleave(BLOCK, 1)
        return w[:, :k]

    for e, rows in routed.items():
        at = torch.tensor([t for t, _ in rows], device="cuda")
        h = x[at] @ weights(s["up"], e, 2 * i, d).T
        h = h[:, :i] * torch.sigmoid(h[:, :i]) * h[:, i:]
        out = h @ weights(s["down"], e, d, i).T
        y.index_add_(0, at, out * torch.tensor([w for _, w in rows], dtype=torch.float64, device="cuda")[:, None])
    return y
