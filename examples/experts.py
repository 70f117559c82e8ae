"""A layer of experts, trained and then served: routing, grouped MXFP4 products and the AdamW step.

Each token takes `top_k` of the experts, and its output is their gated sum.  The experts learn to
give what another set of weights gives.  A whole training step, forward, backward and update, is
one CUDA graph: the experts' sizes stay on the device.  Serving then runs token by token from the
weights' row blob alone.

    python examples/experts.py
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from mxfp4_block_scaled_quantize_gb300 import abi  # noqa: E402
from mxfp4_block_scaled_quantize_gb300.grouped import MXFP4GroupedLinear  # noqa: E402
from mxfp4_block_scaled_quantize_gb300.optim import AdamW  # noqa: E402


def route(x, router, top_k):
    """The tokens' order by expert: offsets [E + 1] and rows [T * top_k] (int32), each token's
    places in that order [T, top_k], and its gates."""
    scores, experts = (x.float() @ router).topk(top_k, dim=1)
    order = torch.sort(experts.reshape(-1), stable=True).indices
    sizes = torch.zeros(router.size(1), dtype=torch.int64, device=x.device)
    sizes.scatter_add_(0, experts.reshape(-1), torch.ones_like(experts.reshape(-1)))
    offsets = torch.zeros(router.size(1) + 1, dtype=torch.int32, device=x.device)
    offsets[1:] = sizes.cumsum(0)
    places = torch.empty_like(order)
    places[order] = torch.arange(order.numel(), device=x.device)
    return offsets, (order // top_k).to(torch.int32), places.view(-1, top_k), scores.softmax(dim=1)


def gather_outputs(y, places, gates):
    """The gated sum of each token's rows of y (grouped order), in fp32 and always in the same order."""
    return (y[places].float() * gates.unsqueeze(2)).sum(1)


def train(tokens=1024, experts=8, n=512, k=512, top_k=2, steps=60, lr=2e-3, seed=0):
    """Losses of all steps, and what serving needs: router, bf16 weights, the last step's inputs."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(tokens, k, device="cuda", generator=g).to(torch.bfloat16)
    router = torch.randn(k, experts, device="cuda", generator=g)
    teacher = torch.randn(experts, n, k, device="cuda", generator=g) / k ** 0.5
    offsets, rows, places, gates = route(x, router, top_k)
    target = torch.zeros(tokens, n, device="cuda")
    for j in range(top_k):
        expert = torch.bucketize(places[:, j].contiguous(), offsets[1:].long(), right=True)
        for e in range(experts):
            own = expert == e
            target[own] += gates[own, j:j + 1] * (x[own].float() @ teacher[e].T)

    master = torch.randn(experts, n, k, device="cuda", generator=g) * (0.1 / k ** 0.5)
    weight = master.to(torch.bfloat16)
    layer = MXFP4GroupedLinear(experts, n, k, tokens * top_k)
    optimizer = AdamW([weight], masters=[master], state_bits=8, lr=lr, weight_decay=0.0, seed=seed)
    dynamic = torch.empty(5, device="cuda")
    gate_rows = torch.empty(tokens * top_k, 1, device="cuda")
    gate_rows[places.reshape(-1)] = gates.reshape(-1, 1)

    def step():
        y = layer.forward(x, weight, offsets, rows)
        error = gather_outputs(y, places, gates) - target
        dy = (error[rows.long()] * gate_rows * (2 / error.numel())).to(torch.bfloat16)
        _, dw = layer.backward(dy, offsets)
        optimizer.step([dw], dynamic=dynamic)
        return error.square().mean()

    def hyperparameters(t):
        b1, b2 = optimizer.betas
        dynamic.copy_(torch.tensor([lr, 1 - b1 ** t, 1 - b2 ** t, 1.0, t]))

    hyperparameters(1)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):   # the first step, outside the graph
        losses = [step().item()]
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        loss = step()
    for t in range(2, steps + 1):
        hyperparameters(t)
        graph.replay()
        losses.append(loss.item())
    return losses, router, weight, x


def serve(x, router, weight, top_k=2):
    """Outputs [T, N] of the tokens of x, one at a time, from the row blob of the weights."""
    experts, n, k = weight.shape
    w_q, w_s = abi.quantize_grouped(weight.view(-1, k), groups=experts, dual=False)[:2]
    layer = MXFP4GroupedLinear(experts, n, k, top_k, train=False)
    out = torch.empty(x.size(0), n, device="cuda")
    for t in range(x.size(0)):
        offsets, rows, places, gates = route(x[t:t + 1], router, top_k)
        y = layer.forward_packed(x[t:t + 1], w_q, w_s, offsets, rows)
        out[t] = gather_outputs(y, places, gates)[0]
    return out


def main():
    losses, router, weight, x = train()
    print(f"loss {losses[0]:.4f} -> {losses[-1]:.4f} in {len(losses)} steps")
    print("served 4 tokens:", tuple(serve(x[:4], router, weight).shape))


if __name__ == "__main__":
    main()
