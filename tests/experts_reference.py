"""The experts' products from their definition in 64 bits, expert by expert, and
elementwise bounds of the library's results.

With p the operands' significant bits, u = 2^-p half a step of their type:

* a product's sum of n terms: the tensor cores' adder truncates by less than 2^-23 of
  the sum a step of 16 products, and sums are added in fp32 after 16 steps (g, u and v
  = grad W_out of a training step: 2^-19 of the sum of magnitudes, and as much again for
  the additions of up to 32 such sums) or 256 steps (everything else: 2^-15);
* h = silu(g) u inherits |silu'| <= 1.1 times g's error and u's, 2^-20 for its
  exponential, division and products, and is rounded to the type (u, or half of
  fp16's smallest step);
* dg = w v u silu'(g), with |silu''| <= 0.5, and du = w v silu(g) likewise; fp16 holds them
  times a power of two that brings the largest |grad| to 16 or more;
* the products that follow add their operands' errors to their own 2^-15, the fp32
  sums over a token's rows 2^-21, and the result is rounded once more;
* bf16: rows on their way to those sums are halves with a power of two of their own, half a
  step of 11 bits: 2^-12 of each.
"""
from __future__ import annotations

import torch

SUM, EXACT_SUM = 2.0 ** -15, 2.0 ** -18


class Experts:
    def __init__(self, x, w_in, w_out, ids, weights, grad=None, exact=None):
        """exact: the sums of g and u are those of a training step (default: where there is a gradient)."""
        T, D = x.shape
        E, _, F = w_in.shape[0], 0, w_out.shape[2]
        unit = torch.finfo(x.dtype).eps / 2
        tiny = 2.0 ** -25 if x.dtype == torch.float16 else 0.0
        row = 2.0 ** -12 if x.dtype == torch.bfloat16 else 0.0
        exact = grad is not None if exact is None else exact
        first = EXACT_SUM if exact else SUM
        f64 = {"dtype": torch.float64, "device": x.device}
        self.out, self.e_out, size = (torch.zeros(T, D, **f64) for _ in range(3))
        if grad is not None:
            self.dx, self.e_dx, size_dx = (torch.zeros(T, D, **f64) for _ in range(3))
            self.dw_in, self.e_dw_in = (torch.zeros(E, 2 * F, D, **f64) for _ in range(2))
            self.dw_out, self.e_dw_out = (torch.zeros(E, D, F, **f64) for _ in range(2))
            self.dw, self.e_dw = (torch.zeros(ids.shape, **f64) for _ in range(2))
            most = float(grad.double().abs().nan_to_num(0.0, 0.0, 0.0).max()) if grad.numel() else 0.0
            small = tiny * most / 16
        for e in range(E):
            t, j = torch.nonzero(ids == e, as_tuple=True)
            if not t.numel():
                continue
            a, b, xe = w_in[e].double(), w_out[e].double(), x[t].double()
            w = weights[t, j].double()[:, None]
            gu, e_gu = xe @ a.t(), first * (xe.abs() @ a.abs().t())
            g, up, e_g, e_u = gu[:, :F], gu[:, F:], e_gu[:, :F], e_gu[:, F:]
            s = torch.sigmoid(g)
            silu = g * s
            h = silu * up
            e_h0 = 1.1 * up.abs() * e_g + silu.abs() * e_u + 2.0 ** -20 * h.abs()
            e_h = e_h0 + unit * h.abs() + tiny
            y = h @ b.t()
            e_y = e_h @ b.abs().t() + SUM * (h.abs() @ b.abs().t()) + row * y.abs()
            self.out.index_add_(0, t, w * y)
            self.e_out.index_add_(0, t, w.abs() * e_y)
            size.index_add_(0, t, w.abs() * y.abs())
            if grad is None:
                continue
            ge = grad[t].double()
            v, e_v = ge @ b, EXACT_SUM * (ge.abs() @ b.abs())
            self.dw[t, j] = (h * v).sum(dim=1)
            self.e_dw[t, j] = (h.abs() * e_v + (e_h0 + 2.0 ** -20 * h.abs()) * v.abs()).sum(dim=1)
            slope = s * (1 + g * (1 - s))
            dg, du = w * v * up * slope, w * v * silu
            e_dg = w.abs() * (e_v * (up * slope).abs() + v.abs() * (slope.abs() * e_u + 0.5 * up.abs() * e_g)) + \
                (unit + 2.0 ** -20) * dg.abs() + 2.0 ** -20 * (w * v * up).abs() + small
            e_du = w.abs() * (e_v * silu.abs() + 1.1 * v.abs() * e_g) + (unit + 2.0 ** -20) * du.abs() + small
            d, e_d = torch.cat([dg, du], dim=1), torch.cat([e_dg, e_du], dim=1)
            self.dx.index_add_(0, t, d @ a)
            self.e_dx.index_add_(0, t, e_d @ a.abs() + SUM * (d.abs() @ a.abs()) + row * (d @ a).abs())
            size_dx.index_add_(0, t, (d @ a).abs())
            self.dw_in[e] = d.t() @ xe
            self.e_dw_in[e] = e_d.t() @ xe.abs() + SUM * (d.abs().t() @ xe.abs())
            e_hw = w.abs() * e_h0 + (unit + 2.0 ** -23) * (w * h).abs() + tiny
            self.dw_out[e] = ge.t() @ (w * h)
            self.e_dw_out[e] = ge.abs().t() @ e_hw + SUM * (ge.abs().t() @ (w * h).abs())
        self.e_out = 1.01 * (self.e_out + 2.0 ** -21 * size + unit * self.out.abs()) + tiny
        if grad is not None:
            self.e_dx = 1.01 * (self.e_dx + 2.0 ** -21 * size_dx + unit * self.dx.abs()) + tiny
            self.e_dw_in = 1.01 * (self.e_dw_in + unit * self.dw_in.abs()) + tiny
            self.e_dw_out = 1.01 * (self.e_dw_out + unit * self.dw_out.abs()) + tiny
            self.e_dw = 1.01 * self.e_dw + 2.0 ** -126

    def check(self, **got):
        """got: out, dx, dw_in, dw_out, dw as computed; each within its bound everywhere."""
        for name, v in got.items():
            want, bound = getattr(self, name), getattr(self, "e_" + name)
            assert v.shape == want.shape, name
            v = v.double()
            assert torch.isfinite(v).all(), f"{name}: not finite"
            off = (v - want).abs()
            ratio = torch.where(off == 0, torch.zeros_like(off), off / bound.clamp_min(1e-300))
            assert ratio.numel() == 0 or float(ratio.max()) <= 1.0, \
                f"{name}: error / bound {float(ratio.max()):.3g} at {int(ratio.argmax())} of {tuple(v.shape)}"
