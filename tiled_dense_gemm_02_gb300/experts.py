"""Operators of a sparse layer (``include/tgemm_experts.h``): the routing of
tokens to experts, and the experts' products.

The first functions carry the names of the C ABI and only marshal arguments;
``route_experts`` and ``route_experts_backward`` take torch tensors (torch
supplies device memory and streams only).
"""
from __future__ import annotations

import ctypes
import functools
import math
from operator import index

from . import BF16, F16, F32, OK, TgemmError, library
from .loss import _current_stream, _guarded, _on_stream, _pitch

ROUTE_MAX_EXPERTS, ROUTE_MAX_K, ROUTE_MAX_GROUPS = 1024, 32, 32  # TGEMM_ROUTE_MAX_*
ROUTE_SOFTMAX, ROUTE_SIGMOID = 0, 1                              # enum tgemm_route_scoring
ROUTE_GROUP_MAX, ROUTE_GROUP_TOP2 = 0, 1                         # enum tgemm_route_group_score

EXPERT_EXPORTS = ("tgemm_route_forward", "tgemm_route_backward")


class RouteOptions(ctypes.Structure):
    """struct tgemm_route_options"""
    _fields_ = [("scoring", ctypes.c_int), ("renormalize", ctypes.c_int), ("scale", ctypes.c_float),
                ("groups", ctypes.c_int), ("top_groups", ctypes.c_int), ("group_score", ctypes.c_int),
                ("reserved", ctypes.c_int * 2)]


def _declare(lib):
    i64, vp, ip = ctypes.c_int64, ctypes.c_void_p, ctypes.c_int
    op = ctypes.POINTER(RouteOptions)
    lib.tgemm_route_forward.argtypes = [i64, i64, i64, vp, i64, ip, vp, op, vp, vp, vp]
    lib.tgemm_route_backward.argtypes = [i64, i64, i64, vp, i64, ip, vp, vp, op, vp, i64, vp]
    for name in EXPERT_EXPORTS:
        getattr(lib, name).restype = ip
    return lib


_lib = _declare(library())


def _opts(options):
    if options is None:
        return None
    if isinstance(options, RouteOptions):
        return ctypes.byref(options)
    o = RouteOptions()
    for k, v in dict(options).items():
        setattr(o, k, v)
    return ctypes.byref(o)


def route_forward(T, E, k, logits, ld, dtype, bias, ids, weights, options=None, stream=0) -> int:
    """tgemm_route_forward: device pointers as ints; returns the status."""
    return _lib.tgemm_route_forward(T, E, k, logits, ld, dtype, bias, _opts(options), ids, weights, stream)


def route_backward(T, E, k, logits, ld, dtype, ids, grad, d_logits, ld_out, options=None, stream=0) -> int:
    """tgemm_route_backward"""
    return _lib.tgemm_route_backward(T, E, k, logits, ld, dtype, ids, grad, _opts(options), d_logits, ld_out, stream)


# ------------------------------------------------------------ torch functions

@functools.lru_cache(maxsize=256)
def _route_options(scoring, renormalize, scale, groups, top_groups, group_score):
    return ctypes.byref(RouteOptions(scoring=scoring, renormalize=renormalize, scale=scale, groups=groups,
                                     top_groups=top_groups, group_score=group_score))


def _choice(name, value, choices):
    if value not in choices:
        raise ValueError(f"{name} must be one of {', '.join(map(repr, choices))}, got {value!r}")
    return choices.index(value)


def _plain(scoring, renormalize, scale, groups=1, top_groups=1, group_score="max"):
    """The options as plain numbers.  The library holds scale in float32, where 0 stands for the default: what rounds to
    0 or to infinity there is refused."""
    factor = ctypes.c_float(float(scale)).value
    if not 0.0 < factor < math.inf:
        raise ValueError(f"scale must be positive within float32's range, got {scale}")
    return (_choice("scoring", scoring, ("softmax", "sigmoid")), int(bool(renormalize)), factor, index(groups),
            index(top_groups), _choice("group_score", group_score, ("max", "top2")))


def _logits(logits):
    """(torch, device, T, E, dtype code, row pitch)"""
    import torch
    if logits.dim() != 2 or logits.shape[1] < 1:
        raise ValueError("logits must be a matrix [T, E]")
    code = {torch.float32: F32, torch.float16: F16, torch.bfloat16: BF16}.get(logits.dtype)
    if code is None:
        raise ValueError(f"unsupported dtype: {logits.dtype}")
    device = logits.get_device()
    if device < 0:
        raise ValueError("logits must be on a CUDA device")
    T, E = logits.shape
    return torch, device, T, E, code, _pitch("logits", logits, T, E)


def _places(name, t, shape, dtype, device):
    """A dense [T, k] tensor."""
    if t.shape != shape or t.dtype != dtype:
        raise ValueError(f"{name} must be {list(shape)} {dtype}, got {list(t.shape)} {t.dtype}")
    if t.get_device() != device:
        raise ValueError(f"{name} must be on the device of the other tensors")
    return t if t.is_contiguous() else t.contiguous()


@functools.cache
def _route_node():
    """The torch function that records a routing whose logits require a gradient."""
    import torch

    class Routing(torch.autograd.Function):
        @staticmethod
        def forward(ctx, logits, top_k, bias, options, more):
            ids, weights = _route(logits, top_k, bias, options)
            ctx.mark_non_differentiable(ids)
            ctx.save_for_backward(logits, ids)
            ctx.more = more
            return ids, weights

        @staticmethod
        @torch.autograd.function.once_differentiable
        def backward(ctx, _, grad):
            logits, ids = ctx.saved_tensors
            return route_experts_backward(logits, ids, grad, **ctx.more), None, None, None, None

    return Routing


def _route(logits, top_k, bias, options):
    torch, device, T, E, code, ld = _logits(logits)
    k = index(top_k)
    if bias is not None:
        if bias.shape != (E,) or bias.dtype != torch.float32 or bias.get_device() != device:
            raise ValueError(f"bias must be a vector of {E} {torch.float32} values on the device of logits")
        bias = bias if bias.is_contiguous() else bias.contiguous()
    ids = torch.empty((T, max(0, k)), dtype=torch.int64, device=logits.device)
    weights = torch.empty((T, max(0, k)), dtype=torch.float32, device=logits.device)
    st = _guarded(torch, device, _lib.tgemm_route_forward,
                  (T, E, k, logits.data_ptr(), ld, code, 0 if bias is None else bias.data_ptr(),
                   _route_options(*options), ids.data_ptr(), weights.data_ptr(), _current_stream(torch, device)))
    if st != OK:
        raise TgemmError(st, "tgemm_route_forward")
    return ids, weights


@_on_stream
def route_experts(logits, top_k, *, scoring="softmax", bias=None, groups=1, top_groups=1, group_score="max",
                  renormalize=True, scale=1.0):
    """The ``top_k`` experts of every row of ``logits`` [T, E] and their weights:
    ``(ids [T, top_k] int64, weights [T, top_k] float32)``, by falling score.

    scoring: "softmax" over the row or "sigmoid" of each logit.  bias [E]
    float32 is added to the scores that experts are picked by, and has no part in
    the weights.  groups > 1: experts come from the ``top_groups`` of ``groups``
    equal groups of neighbours with the largest value, their largest score
    ("max") or the sum of their two largest ("top2").  Weights are the picked
    scores, divided by their sum (renormalize), times scale.

    Of equal scores the lowest index comes first.  A logit of -inf masks its expert;
    where fewer than top_k are left, the rest of the row is id -1, weight 0, which
    the experts' products pass over.  logits in bf16, fp16 or fp32, any row
    stride; up to 1024 experts, 32 picks, 32 groups.

    If logits requires a gradient, so do the weights; the picks have none.
    """
    options = _plain(scoring, renormalize, scale, groups, top_groups, group_score)
    if logits.requires_grad or (bias is not None and bias.requires_grad):
        import torch
        if torch.is_grad_enabled() and bias is not None and bias.requires_grad:
            raise ValueError("bias gets no gradient: detach it")
        if torch.is_grad_enabled():
            return _route_node().apply(logits, top_k, bias, options,
                                       {"scoring": scoring, "renormalize": renormalize, "scale": scale})
    return _route(logits, top_k, bias, options)


@_on_stream
def route_experts_backward(logits, ids, grad_weights, *, scoring="softmax", renormalize=True, scale=1.0):
    """The gradient of ``sum(grad_weights * weights)`` with respect to
    ``logits``, [T, E] in its type, for ``ids`` and the options of the forward
    call.  It is outside torch's graph."""
    options = _plain(scoring, renormalize, scale)
    torch, device, T, E, code, ld = _logits(logits)
    if ids.dim() != 2:
        raise ValueError("ids must be a matrix [T, top_k]")
    shape = torch.Size((T, ids.shape[1]))
    ids = _places("ids", ids, shape, torch.int64, device)
    grad_weights = _places("grad_weights", grad_weights, shape, torch.float32, device)
    out = torch.empty((T, E), dtype=logits.dtype, device=logits.device)
    st = _guarded(torch, device, _lib.tgemm_route_backward,
                  (T, E, shape[1], logits.data_ptr(), ld, code, ids.data_ptr(), grad_weights.data_ptr(),
                   _route_options(*options), out.data_ptr(), E, _current_stream(torch, device)))
    if st != OK:
        raise TgemmError(st, "tgemm_route_backward")
    return out
