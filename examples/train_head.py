"""Train a vocabulary head on tokens and on a teacher's stored top logits.

A frozen teacher head labels random hidden states: each token gets a sampled
target, and the teacher's K largest logits with their entries, as a store of
teacher outputs would hold them.  The student head starts elsewhere and takes
plain gradient steps on

    mean cross entropy + weight * temperature^2 * mean divergence from the teacher

through the library's two losses, whose logits are never written out: both
return one loss per token and, from its gradient, those of the hidden states and
of the head.  A tenth of the tokens is padding (ignored, its hidden states never
written).

    python examples/train_head.py [--tokens 512] [--vocab 8192] [--depth 256] [--steps 30]
"""
from __future__ import annotations

import argparse
import math
import os
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)


def head_loss(hidden, weight, targets, ids, logits, temperature, mix):
    """(cross entropy, divergence, d_hidden, d_weight) of the training loss: means over the tokens that count."""
    import tiled_dense_gemm_02_gb300 as tg
    n = (targets >= 0).sum().clamp_min(1)
    grad = (targets >= 0).float() / n
    xent, lse = tg.linear_cross_entropy(hidden, weight, targets)
    dh, dw = tg.linear_cross_entropy_backward(hidden, weight, targets, lse, grad)
    kl, lse_t = tg.linear_distillation(hidden, weight, ids, logits, temperature=temperature)
    dh_t, dw_t = tg.linear_distillation_backward(hidden, weight, ids, logits, lse_t, mix * temperature ** 2 * grad,
                                                 temperature=temperature)
    return xent.sum() / n, kl.sum() / n, dh.float() + dh_t, dw.float() + dw_t


def train(tokens=512, vocab=8192, depth=256, top=16, steps=30, rate=8.0, temperature=2.0, mix=0.5, seed=0,
          dtype=None, report=None):
    """The training losses, step by step; report(step, cross entropy, divergence) is called for each."""
    import torch
    dtype = dtype or torch.bfloat16
    gen = torch.Generator(device="cuda").manual_seed(seed)
    hidden = torch.randn(tokens, depth, device="cuda", generator=gen).to(dtype)
    teacher = torch.randn(vocab, depth, device="cuda", generator=gen) * (3.0 / math.sqrt(depth))
    z = hidden.float() @ teacher.t()
    logits, ids = z.topk(top, dim=1)
    targets = torch.multinomial(z.softmax(dim=1), 1, generator=gen)[:, 0]
    padding = torch.rand(tokens, device="cuda", generator=gen) < 0.1
    targets[padding] = -100
    ids[padding] = -1
    hidden[padding] = float("nan")
    master = torch.randn(vocab, depth, device="cuda", generator=gen) * (0.5 / math.sqrt(depth))  # fp32 weights
    history = []
    for step in range(steps):
        xent, kl, dh, dw = head_loss(hidden, master.to(dtype), targets, ids, logits, temperature, mix)
        master -= rate * dw
        history.append((float(xent), float(kl), float(dh.norm()), float(dw.norm())))
        if report:
            report(step, *history[-1])
    return history


def main():
    p = argparse.ArgumentParser(description=__doc__.split("\n\n")[0])
    p.add_argument("--tokens", type=int, default=512)
    p.add_argument("--vocab", type=int, default=8192)
    p.add_argument("--depth", type=int, default=256)
    p.add_argument("--steps", type=int, default=30)
    a = p.parse_args()
    train(a.tokens, a.vocab, a.depth, steps=a.steps,
          report=lambda i, x, k, dh, dw: print(f"step {i:3d}  cross entropy {x:7.4f}  divergence {k:7.4f}  "
                                               f"|dH| {dh:.3g}  |dW| {dw:.3g}"))


if __name__ == "__main__":
    main()
