"""Routing from its definition in 64 bits, and the tolerances of the library's
weights and gradients.

Picks are whole numbers and have to be equal.  A weight in fp32: the
exponential of x - m (x the picked logit, m the row's largest, R the largest
|x - m| of the row) is off by two last bits, 4 u with u = 2^-24, and by u R through
the rounding of x - m; the sum of E such terms by as much again and by u per
addition of a chain (E / 32 in a lane, 5 between lanes); division, scale and
storing by u each.  Together u (16 + E / 32 + 2 R), relative; sigmoids by less.  A
gradient is scale p (g - sum g p), p such a share, so it inherits four of
these (two shares, their sum, 1 - s) times scale p (|g| + sum |g| p), and
half a step of its type.
"""
from __future__ import annotations

import math

import torch

U = 2.0 ** -24
SMALLEST = {torch.bfloat16: 2.0 ** -126, torch.float16: 2.0 ** -24, torch.float32: 2.0 ** -126}


def first_largest(v):
    """Index of each row's largest value, the lowest of several; NaN is the largest."""
    at = torch.arange(v.shape[1], device=v.device).expand_as(v)
    nan = v != v
    top = torch.where(nan.any(dim=1), torch.full_like(v[:, 0], math.nan), v.amax(dim=1))[:, None]
    hit = torch.where(nan.any(dim=1)[:, None], nan, v == top)
    return torch.where(hit, at, torch.full_like(at, v.shape[1])).amin(dim=1).clamp_max(v.shape[1] - 1)


class Routed:
    def __init__(self, logits, k, scoring="softmax", bias=None, groups=1, top_groups=1, group_score="max",
                 renormalize=True, scale=1.0):
        x = logits.double()
        T, E = x.shape
        self.E, self.k, self.scale, self.sigmoid, self.renormalize = E, k, scale, scoring == "sigmoid", renormalize
        low = torch.full_like(x, -math.inf)
        masked = x == -math.inf
        m = torch.where(masked.all(dim=1, keepdim=True), torch.zeros_like(x[:, :1]), x.amax(dim=1, keepdim=True))
        if self.sigmoid:
            self.score = 1 / (1 + torch.exp(-x))
        else:
            e = torch.exp(x - m)
            total = e.sum(dim=1, keepdim=True)
            self.score = torch.where(total == 0, torch.zeros_like(e), e / total)
        self.range = torch.where(masked, torch.zeros_like(x), (x - m).abs()).nan_to_num(posinf=0.0).amax(dim=1, keepdim=True)
        key = torch.where(masked, low, self.score if bias is None else self.score + bias.double())
        if bias is None and (groups == 1 or group_score == "max"):
            key = x  # logits in their own order
        if groups > 1:
            size = E // groups
            part = key.reshape(T * groups, size)
            value = part.amax(dim=1)
            if group_score == "top2" and size > 1:
                rest = part.scatter(1, first_largest(part)[:, None], -math.inf).amax(dim=1)
                value = torch.where(rest > -math.inf, value + rest, value)
            value = value.view(T, groups)
            keep = torch.zeros_like(value, dtype=torch.bool)
            for _ in range(top_groups):
                at = first_largest(value)[:, None]
                keep |= torch.zeros_like(keep).scatter_(1, at, value.gather(1, at) > -math.inf)
                value = value.scatter(1, at, -math.inf)
            key = torch.where(keep.repeat_interleave(size, dim=1), key, low)
        ids = []
        for _ in range(k):
            at = first_largest(key)
            v = key.gather(1, at[:, None])[:, 0]
            ids.append(torch.where(v == -math.inf, torch.full_like(at, -1), at))
            key = key.scatter(1, at[:, None], -math.inf)
        self.ids = torch.stack(ids, dim=1)
        self.used = self.ids >= 0
        zero = torch.zeros((), dtype=x.dtype, device=x.device)
        p = torch.where(self.used, self.score.gather(1, self.ids.clamp_min(0)), zero)
        if renormalize:
            # from logarithms: sigmoids of very negative logits underflow
            log = torch.where(self.sigmoid_of(x), torch.nn.functional.logsigmoid(x), x).gather(1, self.ids.clamp_min(0))
            log = torch.where(self.used, log, torch.full_like(log, -math.inf))
            top = torch.where(self.used.any(dim=1, keepdim=True), log.amax(dim=1, keepdim=True), torch.zeros_like(log[:, :1]))
            e = torch.exp(log - top)
            p = torch.where(self.used, e / e.sum(dim=1, keepdim=True), zero)
        self.share = p
        self.weights = scale * p
        self.rel = U * (16 + E / 32 + 2 * self.range)

    def sigmoid_of(self, x):
        return torch.full((1, 1), self.sigmoid, device=x.device)

    def check(self, ids, weights):
        assert torch.equal(ids, self.ids)
        assert weights.dtype == torch.float32 and bool((weights[~self.used] == 0).all())
        off = (weights.double() - self.weights).abs()
        assert bool((off <= self.rel * self.weights + 2.0 ** -126).all()), float((off / (self.rel * self.weights).clamp_min(1e-300)).max())

    def check_gradient(self, got, g):
        zero = torch.zeros_like(self.share)
        g = torch.where(self.used, g.double(), zero)
        at = self.ids.clamp_min(0)
        picked = torch.where(self.used, self.score.gather(1, at), zero)
        if self.renormalize:
            d = self.share * (g - (g * self.share).sum(dim=1, keepdim=True))
            size = self.share * (g.abs() + (g.abs() * self.share).sum(dim=1, keepdim=True))
            if self.sigmoid:
                d, size = d * (1 - picked), size * (1 - picked)
        elif self.sigmoid:
            d = g * picked * (1 - picked)
            size = d.abs()
        else:
            d, size = g * picked, g.abs() * picked
        want = torch.zeros_like(self.score).scatter_add_(1, at, d)
        most = torch.zeros_like(self.score).scatter_add_(1, at, size)
        if not self.renormalize and not self.sigmoid:
            want = want - self.score * d.sum(dim=1, keepdim=True)
            most = most + self.score * size.sum(dim=1, keepdim=True)
        want, most = self.scale * want, self.scale * most
        bound = 4 * self.rel * most + torch.finfo(got.dtype).eps / 2 * want.abs() + SMALLEST[got.dtype]
        off = (got.double() - want).abs()
        assert bool((off <= bound).all()), float((off / bound).max())
