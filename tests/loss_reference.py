"""The vocabulary-head losses from their definition in 64 bits, on whole
logits, and the tolerances of the library's results.

Every bound follows from the roundings that the computation makes, elementwise:

* a logit is a sum of D products held in fp32.  Its rounding errors add up like
  a random walk: |dz| <= E = 4 sqrt(D) 2^-23 S, with S the row's largest sum of
  |h w| times the scale, and 4 for the tail over many logits;
* lse and the loss inherit E and are themselves fp32 sums of values of the size
  of lse: another 2^-20 (1 + |lse|) covers the exponentials' and the sums'
  roundings;
* a probability inherits E + 2^-22 (1 + |lse|) as a relative error, and is 0
  below fp32's smallest normal number, 2^-126;
* dz is rounded to the operands' type (2^-p relative, p its significant bits: 8
  for bf16, 11 for fp16, 24 for fp32), the products that follow hold fp32 sums (as above, relative
  to the sum of magnitudes), and the result is rounded once more.
"""
from __future__ import annotations

import math

import torch

import workloads as wl

UNIT = {t: 2.0 ** -wl.FORMATS[f][0] for t, f in ((torch.bfloat16, "bf16"), (torch.float16, "f16"),
                                                 (torch.float32, "f32"))}
# half the spacing of the smallest numbers of the output type
TINY = {torch.bfloat16: 0.0, torch.float16: 2.0 ** -25, torch.float32: 0.0}


class Reference:
    """loss, lse, dh, dw in float64 and e_loss, e_lse, e_dh, e_dw, their elementwise bounds."""

    def __init__(self, h, w, counts, q, own, scale=1.0, z_loss=0.0, g=None):
        """q [T, V] float64: the target distribution (zero rows where not counts)."""
        T, D = h.shape
        h64 = torch.where(counts[:, None], h.double(), torch.zeros((), dtype=torch.float64, device=h.device))
        w64 = w.double()
        z = scale * (h64 @ w64.t())
        size = scale * (h64.abs() @ w64.abs().t()).amax(dim=1)
        lse = torch.logsumexp(z, dim=1)
        dot = (q * z).sum(dim=1)
        zero = torch.zeros_like(lse)
        self.loss = torch.where(counts, own + lse - dot + z_loss * lse ** 2, zero)
        self.lse = torch.where(counts, lse, zero)
        e_z = 4 * math.sqrt(D) * 2.0 ** -23 * size
        self.e_lse = e_z + 2.0 ** -20 * (1 + lse.abs())
        self.e_loss = 2 * e_z * (1 + 2 * z_loss * lse.abs()) + 2.0 ** -19 * (1 + lse.abs() + z_loss * lse ** 2 +
                                                                            own.abs() + (q * z).abs().sum(dim=1))
        if g is None:
            return
        p = torch.exp(z - lse[:, None])
        c = torch.where(counts, g.double(), zero)[:, None]
        cp = 1 + 2 * z_loss * lse[:, None]
        dz = c * (cp * p - q) * scale
        mass = c.abs() * (cp * p + q) * scale
        u = UNIT[h.dtype]
        e_p = (e_z + 2.0 ** -22 * (1 + lse.abs()))[:, None]
        e_dz = mass * e_p + dz.abs() * u + mass * 2.0 ** -22 + c.abs() * scale * 2.0 ** -126
        self.dh, self.dw = dz @ w64, dz.t() @ h64
        V = w.shape[0]
        self.e_dh = 1.01 * (e_dz @ w64.abs() + 4 * math.sqrt(V) * 2.0 ** -23 * (mass @ w64.abs()) +
                            u * self.dh.abs()) + TINY[h.dtype]
        self.e_dw = 1.01 * (e_dz.t() @ h64.abs() + 4 * math.sqrt(T) * 2.0 ** -23 * (mass.t() @ h64.abs()) +
                            u * self.dw.abs()) + TINY[h.dtype]

    def check(self, **got):
        """got: loss, lse, dh, dw as computed; each within its bound everywhere."""
        for name, x in got.items():
            want, bound = getattr(self, name), getattr(self, "e_" + name)
            assert x.shape == want.shape, name
            x = x.double()
            assert torch.isfinite(x).all(), f"{name}: not finite"
            ratio = (x - want).abs() / bound.clamp_min(1e-300)
            ratio = torch.where(x == want, torch.zeros_like(ratio), ratio)
            assert ratio.numel() == 0 or float(ratio.max()) <= 1.0, \
                f"{name}: error / bound {float(ratio.max()):.3g} at {int(ratio.argmax())} of {tuple(x.shape)}"


def xent(h, w, targets, ignore_index=-100, scale=1.0, smoothing=0.0, z_loss=0.0, g=None):
    T, V = h.shape[0], w.shape[0]
    counts = targets != ignore_index
    q = torch.full((T, V), smoothing / V, dtype=torch.float64, device=h.device)
    q[torch.arange(T, device=h.device), torch.where(counts, targets, torch.zeros_like(targets))] += 1 - smoothing
    q = q * counts[:, None]
    return Reference(h, w, counts, q, torch.zeros(T, dtype=torch.float64, device=h.device), scale, z_loss, g)


def distill(h, w, ids, logits, temperature=1.0, g=None):
    T, V = h.shape[0], w.shape[0]
    t = logits.double() / temperature
    t = torch.where(ids >= 0, t, torch.full_like(t, -math.inf))
    counts = (t > -math.inf).any(dim=1)
    top = torch.where(counts, t.amax(dim=1), torch.zeros(T, dtype=torch.float64, device=h.device))
    e = torch.exp(t - top[:, None])
    total = torch.where(counts, e.sum(dim=1), torch.ones_like(top))
    mass = e / total[:, None]
    own = torch.special.xlogy(mass, mass).sum(dim=1)
    q = torch.zeros(T, V, dtype=torch.float64, device=h.device)
    q.scatter_add_(1, ids.clamp_min(0), mass)
    # an unused place adds 0 to entry 0
    return Reference(h, w, counts, q, own, 1.0 / temperature, 0.0, g)
