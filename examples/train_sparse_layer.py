"""Train a sparse layer: a router, a few experts a token, gradients clipped by their norm.

A dense teacher maps random hidden states to targets; a router and its experts learn
them by plain gradient steps.  Every step is

    logits = hidden @ router.T                    (tgemm's plain product)
    ids, weights = route_experts(logits, top_k)   (a bias keeps the experts' load even)
    out = expert_mlp(hidden, w_in, w_out, ids, weights)

then the backward calls of both, and clip_gradients over all of the step's gradients.
The bias follows the load: an expert with more rows than its share loses a little,
the others win a little; it decides picks and has no part in the weights.

    python examples/train_sparse_layer.py [--tokens 2048] [--depth 256] [--experts 8] [--steps 30]
"""
from __future__ import annotations

import argparse
import math
import os
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)


def step(hidden, target, router, w_in, w_out, bias, top_k, limit):
    """(loss, norm, ids, gradients of the router, of w_in and of w_out): the mean square error's, clipped."""
    import torch

    import tiled_dense_gemm_02_gb300 as tg
    logits = tg.matmul(hidden, router.t().contiguous(), out_dtype=torch.float32)
    ids, weights = tg.route_experts(logits, top_k, scoring="sigmoid", bias=bias)
    out, saved = tg.expert_mlp(hidden, w_in, w_out, ids, weights, save=True)
    error = out.float() - target
    loss = error.square().mean()
    grad = (error * (2.0 / error.numel())).to(hidden.dtype)
    _, d_in, d_out, d_weights = tg.expert_mlp_backward(hidden, w_in, w_out, ids, weights, saved, grad, want_hidden=False)
    d_logits = tg.route_experts_backward(logits, ids, d_weights, scoring="sigmoid")
    d_router = tg.matmul(d_logits.to(hidden.dtype).t().contiguous(), hidden, out_dtype=torch.float32)
    grads = [d_router, d_in, d_out]
    return loss, tg.clip_gradients(grads, limit), ids, grads


def train(tokens=2048, depth=256, width=128, experts=8, top_k=2, steps=30, rate=2.0, limit=0.05, seed=0, dtype=None,
          report=None):
    """[(loss, gradient norm, largest share of one expert)], step by step; report(step, ...) is called for each."""
    import torch
    dtype = dtype or torch.bfloat16
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, device="cuda", generator=gen)

    hidden = normal(tokens, depth).to(dtype)
    target = torch.tanh(hidden.float() @ (normal(depth, depth) / math.sqrt(depth)))
    masters = [0.1 * normal(experts, depth), normal(experts, 2 * width, depth) / math.sqrt(depth),
               normal(experts, depth, width) / math.sqrt(width)]
    bias = torch.zeros(experts, device="cuda")
    history = []
    for i in range(steps):
        loss, norm, ids, grads = step(hidden, target, *[m.to(dtype) for m in masters], bias, top_k, limit)
        for master, grad in zip(masters, grads):
            master -= rate * grad
        load = torch.bincount(ids.flatten(), minlength=experts).float()
        bias += 0.01 * torch.sign(load.mean() - load)
        history.append((float(loss), float(norm), float(load.max() / load.sum())))
        if report:
            report(i, *history[-1])
    return history


def main():
    p = argparse.ArgumentParser(description=__doc__.split("\n\n")[0])
    p.add_argument("--tokens", type=int, default=2048)
    p.add_argument("--depth", type=int, default=256)
    p.add_argument("--experts", type=int, default=8)
    p.add_argument("--steps", type=int, default=30)
    a = p.parse_args()
    train(a.tokens, a.depth, experts=a.experts, steps=a.steps,
          report=lambda i, x, n, s: print(f"step {i:3d}  loss {x:7.4f}  |gradient| {n:.3g}  largest expert {s:.0%}"))


if __name__ == "__main__":
    main()
