"""The experts' products at the ends of the numbers' range: their definition in 64 bits with elementwise
bounds that follow each expert's own numbers.

With u half a step of the operands' type (eps / 2, relative: bf16 2^-8, fp16 2^-11):

* a tensor-core sum of n terms is off by 2^-23 of the sum of magnitudes for each of the `steps` truncating steps
  (16 terms) of a chunk, and by 2^-24 for each addition of a chunk;
* g and u inherit that, h = silu(g) u as in tests/experts_reference.py (|silu'| <= 1.1, |silu''| <= 0.5, 2^-20 for its
  exponential, division and products);
* fp16's dg, du and w h are rounded with a power of two of their expert that brings the largest finite one to 2^14 or more:
  half of the smallest step, 2^-25, is then 2^-39 of the largest;
* bf16 rows on their way to a token's sum are halves, off by 2^-11 of each, or bf16, off by 2^-8, where an element of the
  same 32 is smaller than 2^-27 of the largest (2^-28 in the kernel, by the leading powers);
* every output is rounded once.
"""
from __future__ import annotations

import math

import torch


def sum_bound(n, steps):
    return steps * 2.0 ** -23 + math.ceil(n / (16 * steps)) * 2.0 ** -24


def finite_most(*tensors):
    return max(float(t.abs().nan_to_num(0.0, 0.0, 0.0).max()) if t.numel() else 0.0 for t in tensors)


def row_bound(y):
    """The relative error of bf16 rows y [n, D] on their way to the sum, elementwise."""
    n, D = y.shape
    pad = -D % 32
    blocks = torch.nn.functional.pad(y.abs().nan_to_num(0.0, 0.0, 0.0), (0, pad)).view(n, -1, 32)
    most = blocks.amax(dim=2, keepdim=True)
    spread = ((blocks > 0) & (blocks < 2.0 ** -27 * most)).any(dim=2, keepdim=True)
    return torch.where(spread, 2.0 ** -8, 2.0 ** -11).expand_as(blocks).reshape(n, -1)[:, :D]


class Numbers:
    def __init__(self, x, w_in, w_out, ids, weights, grad, train=True):
        """train: the forward call kept g and u (exact sums)."""
        T, D = x.shape
        E, F = w_in.shape[0], w_out.shape[2]
        half = x.dtype == torch.float16
        unit, least = torch.finfo(x.dtype).eps / 2, 2.0 ** -25 if half else 2.0 ** -134
        exact = 12 if half else 16
        f64 = {"dtype": torch.float64, "device": x.device}
        self.out, self.e_out, size, self.dx, self.e_dx, size_dx = (torch.zeros(T, D, **f64) for _ in range(6))
        self.dw_in, self.e_dw_in = (torch.zeros(E, 2 * F, D, **f64) for _ in range(2))
        self.dw_out, self.e_dw_out = (torch.zeros(E, D, F, **f64) for _ in range(2))
        self.dw, self.e_dw = (torch.zeros(ids.shape, **f64) for _ in range(2))
        for e in range(E):
            t, j = torch.nonzero(ids == e, as_tuple=True)
            n = t.numel()
            if not n:
                continue
            a, b, xe, ge = w_in[e].double(), w_out[e].double(), x[t].double(), grad[t].double()
            w = weights[t, j].double()[:, None]
            gu, e_gu = xe @ a.t(), sum_bound(D, exact if train else 256) * (xe.abs() @ a.abs().t())
            g, up, e_g, e_u = gu[:, :F], gu[:, F:], e_gu[:, :F], e_gu[:, F:]
            s = torch.sigmoid(g)
            silu, slope = g * s, s * (1 + g * (1 - s))
            h = silu * up
            e_h0 = 1.1 * up.abs() * e_g + silu.abs() * e_u + 2.0 ** -20 * h.abs()
            e_h = e_h0 + unit * h.abs() + least
            y = h @ b.t()
            e_y = e_h @ b.abs().t() + sum_bound(F, 256) * (h.abs() @ b.abs().t())
            e_y = e_y + (0.0 if half else row_bound(y) * y.abs())
            self.out.index_add_(0, t, w * y)
            self.e_out.index_add_(0, t, w.abs() * e_y)
            size.index_add_(0, t, w.abs() * y.abs())
            v, e_v = ge @ b, sum_bound(D, exact) * (ge.abs() @ b.abs())
            self.dw[t, j] = (h * v).sum(dim=1)
            self.e_dw[t, j] = (h.abs() * e_v + (e_h0 + 2.0 ** -20 * h.abs()) * v.abs()).sum(dim=1)
            dg, du, wh = w * v * up * slope, w * v * silu, w * h
            small, small_h = (2.0 ** -38.9 * finite_most(dg, du), 2.0 ** -38.9 * finite_most(wh)) if half else (0.0, 0.0)
            e_dg = w.abs() * (e_v * (up * slope).abs() + v.abs() * (slope.abs() * e_u + 0.5 * up.abs() * e_g)) + \
                (unit + 2.0 ** -20) * dg.abs() + 2.0 ** -20 * (w * v * up).abs() + small
            e_du = w.abs() * (e_v * silu.abs() + 1.1 * v.abs() * e_g) + (unit + 2.0 ** -20) * du.abs() + small
            d, e_d = torch.cat([dg, du], dim=1), torch.cat([e_dg, e_du], dim=1)
            row = d @ a
            e_row = e_d @ a.abs() + sum_bound(2 * F, 256) * (d.abs() @ a.abs()) + (0.0 if half else row_bound(row) * row.abs())
            self.dx.index_add_(0, t, row)
            self.e_dx.index_add_(0, t, e_row)
            size_dx.index_add_(0, t, row.abs())
            self.dw_in[e] = d.t() @ xe
            self.e_dw_in[e] = e_d.t() @ xe.abs() + sum_bound(n, 256) * (d.abs().t() @ xe.abs())
            e_wh = w.abs() * e_h0 + (unit + 2.0 ** -23) * wh.abs() + small_h
            self.dw_out[e] = ge.t() @ wh
            self.e_dw_out[e] = ge.abs().t() @ e_wh + sum_bound(n, 256) * (ge.abs().t() @ wh.abs())
        adds = ids.shape[1] * 2.0 ** -23
        self.e_out = 1.01 * (self.e_out + adds * size + unit * self.out.abs()) + least
        self.e_dx = 1.01 * (self.e_dx + adds * size_dx + unit * self.dx.abs()) + least
        self.e_dw_in = 1.01 * (self.e_dw_in + unit * self.dw_in.abs()) + least
        self.e_dw_out = 1.01 * (self.e_dw_out + unit * self.dw_out.abs()) + least
        self.e_dw = 1.01 * self.e_dw + 2.0 ** -126

    def check(self, rows=None, experts=None, **got):
        """got: out, dx, dw_in, dw_out, dw; each finite and within its bound, in the given rows or experts (default: all)."""
        for name, v in got.items():
            at = experts if name in ("dw_in", "dw_out") else rows
            want, bound, v = getattr(self, name), getattr(self, "e_" + name), v.double()
            assert v.shape == want.shape, name
            if at is not None:
                want, bound, v = want[at], bound[at], v[at]
            assert bool(torch.isfinite(v).all()), f"{name}: {int((~torch.isfinite(v)).sum())} of {v.numel()} not finite"
            ratio = (v - want).abs() / bound
            assert ratio.numel() == 0 or float(ratio.max()) <= 1.0, \
                f"{name}: error / bound {float(ratio.max()):.3g} at {int(ratio.argmax())} of {tuple(v.shape)}"
