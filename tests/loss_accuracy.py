"""How exact the fp32 losses are as a whole: errors in the norm of a result,
against the definition in 64 bits.

Elementwise bounds that hold for every input (loss_reference.py) are far above
what fp32 arithmetic leaves: a missing bf16 plane of an operand stays inside
them.  In the norm, for operands of mixed signs and logits that spread with a
deviation of about 1:

* a truncating step of the tensor cores' adder takes 0.15 units of 2^-23 at most
  on average, and 32 of them stand behind a sum: 5.7e-7 of a logit, and the same
  of a gradient's sum;
* a probability inherits the logit's error, of a size of about 1, and that of its
  exponential, 2^-22.

Together 1.4e-6, and NORM leaves a tenth for the roundings of the sums.  Two
planes of each operand leave 2^-17 of every product: 2.6e-6 and more of dH and dW.
"""
from __future__ import annotations

import math

import torch

NORM = 1.5e-6


def operands(T, V, D, device, seed=0):
    gen = torch.Generator(device=device).manual_seed(300 + seed)
    h = torch.randn(T, D, device=device, generator=gen)
    w = torch.randn(V, D, device=device, generator=gen) / math.sqrt(D)
    y = torch.randint(0, V, (T,), device=device, generator=gen)
    return h, w, y, torch.rand(T, device=device, generator=gen) / T


def definition(h, w, y, g, product=None):
    """loss, lse, dh, dw of the cross entropy in float64; product(a, b): a b^T as something else computes it."""
    product = product or (lambda a, b: a.double() @ b.double().t())
    z = product(h, w)
    lse = torch.logsumexp(z, dim=1)
    dz = torch.exp(z - lse[:, None])
    dz[torch.arange(len(y)), y] -= 1
    dz *= g.double()[:, None]
    return {"loss": lse - z.gather(1, y[:, None])[:, 0], "lse": lse, "dh": product(dz, w.t()), "dw": product(dz.t(), h.t())}


def check(want, got):
    for name, x in got.items():
        error = float((x.double() - want[name]).norm() / want[name].norm())
        assert error <= NORM, f"{name}: {error:.3g} of its norm off"
