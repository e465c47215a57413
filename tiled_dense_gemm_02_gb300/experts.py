"""Operators of a sparse layer (``include/tgemm_experts.h``): the routing of
tokens to experts, and the experts' products.

The first functions carry the names of the C ABI and only marshal arguments;
``route_experts``, ``expert_mlp`` and their ``_backward`` take torch tensors
(torch supplies device memory and streams only).
"""
from __future__ import annotations

import ctypes
import functools
import math
from operator import index

from . import BF16, F16, F32, OK, TgemmError, library
from .loss import _current_stream, _guarded, _no_tangents, _on_stream, _pitch

ROUTE_MAX_EXPERTS, ROUTE_MAX_K, ROUTE_MAX_GROUPS = 1024, 32, 32  # TGEMM_ROUTE_MAX_*
ROUTE_SOFTMAX, ROUTE_SIGMOID = 0, 1                              # enum tgemm_route_scoring
ROUTE_GROUP_MAX, ROUTE_GROUP_TOP2 = 0, 1                         # enum tgemm_route_group_score

MAX_EXPERTS = 1024                                               # of the products

EXPERT_EXPORTS = ("tgemm_route_forward", "tgemm_route_backward", "tgemm_experts_workspace_size",
                  "tgemm_experts_saved_size", "tgemm_experts_forward", "tgemm_experts_backward")


class RouteOptions(ctypes.Structure):
    """struct tgemm_route_options"""
    _fields_ = [("scoring", ctypes.c_int), ("renormalize", ctypes.c_int), ("scale", ctypes.c_float),
                ("groups", ctypes.c_int), ("top_groups", ctypes.c_int), ("group_score", ctypes.c_int),
                ("reserved", ctypes.c_int * 2)]


class ExpertsOptions(ctypes.Structure):
    """struct tgemm_experts_options"""
    _fields_ = [("wait_timeout_us", ctypes.c_int), ("reserved", ctypes.c_int * 3)]


def _declare(lib):
    i64, vp, ip, sz = ctypes.c_int64, ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
    op, eo, sizes = ctypes.POINTER(RouteOptions), ctypes.POINTER(ExpertsOptions), [ctypes.c_int64] * 5
    lib.tgemm_experts_workspace_size.argtypes = [ip] + sizes + [vp, i64, vp, i64, ip, ctypes.POINTER(sz)]
    lib.tgemm_experts_saved_size.argtypes = sizes + [ip, ctypes.POINTER(sz)]
    lib.tgemm_experts_forward.argtypes = sizes + [vp, i64, vp, i64, vp, i64, vp, vp, ip, eo, vp, i64, vp, sz, vp, sz, vp]
    lib.tgemm_experts_backward.argtypes = sizes + [vp, i64, vp, i64, vp, i64, vp, vp, sz, vp, i64, ip, eo, vp, i64, vp,
                                                   i64, vp, i64, vp, vp, sz, vp]
    lib.tgemm_route_forward.argtypes = [i64, i64, i64, vp, i64, ip, vp, op, vp, vp, vp]
    lib.tgemm_route_backward.argtypes = [i64, i64, i64, vp, i64, ip, vp, vp, op, vp, i64, vp]
    for name in EXPERT_EXPORTS:
        getattr(lib, name).restype = ip
    return lib


_lib = _declare(library())


def _opts(options, kind=RouteOptions):
    if options is None:
        return None
    if isinstance(options, kind):
        return ctypes.byref(options)
    o = kind()
    for k, v in dict(options).items():
        setattr(o, k, v)
    return ctypes.byref(o)


def route_forward(T, E, k, logits, ld, dtype, bias, ids, weights, options=None, stream=0) -> int:
    """tgemm_route_forward: device pointers as ints; returns the status."""
    return _lib.tgemm_route_forward(T, E, k, logits, ld, dtype, bias, _opts(options), ids, weights, stream)


def route_backward(T, E, k, logits, ld, dtype, ids, grad, d_logits, ld_out, options=None, stream=0) -> int:
    """tgemm_route_backward"""
    return _lib.tgemm_route_backward(T, E, k, logits, ld, dtype, ids, grad, _opts(options), d_logits, ld_out, stream)


def experts_workspace_size(backward, T, E, k, D, F, w_in, ld_in, w_out, ld_out, dtype):
    """tgemm_experts_workspace_size: (status, bytes); needs no GPU."""
    n = ctypes.c_size_t(0)
    st = _lib.tgemm_experts_workspace_size(int(backward), T, E, k, D, F, w_in, ld_in, w_out, ld_out, dtype,
                                           ctypes.byref(n))
    return st, n.value


def experts_saved_size(T, E, k, D, F, dtype):
    """tgemm_experts_saved_size: (status, bytes); needs no GPU."""
    n = ctypes.c_size_t(0)
    st = _lib.tgemm_experts_saved_size(T, E, k, D, F, dtype, ctypes.byref(n))
    return st, n.value


def experts_forward(T, E, k, D, F, x, ldx, w_in, ld_in, w_out, ld_out, ids, weights, dtype, out, ldo, saved=0,
                    saved_bytes=0, options=None, workspace=0, workspace_bytes=0, stream=0) -> int:
    """tgemm_experts_forward: device pointers as ints; returns the status."""
    return _lib.tgemm_experts_forward(T, E, k, D, F, x, ldx, w_in, ld_in, w_out, ld_out, ids, weights, dtype,
                                      _opts(options, ExpertsOptions), out, ldo, saved, saved_bytes, workspace,
                                      workspace_bytes, stream)


def experts_backward(T, E, k, D, F, x, ldx, w_in, ld_in, w_out, ld_out, weights, saved, saved_bytes, grad, ldg, dtype,
                     dx, lddx, dw_in, ldd_in, dw_out, ldd_out, d_weights, options=None, workspace=0, workspace_bytes=0,
                     stream=0) -> int:
    """tgemm_experts_backward: outputs that are not wanted may be 0."""
    return _lib.tgemm_experts_backward(T, E, k, D, F, x, ldx, w_in, ld_in, w_out, ld_out, weights, saved, saved_bytes,
                                       grad, ldg, dtype, _opts(options, ExpertsOptions), dx, lddx, dw_in, ldd_in, dw_out,
                                       ldd_out, d_weights, workspace, workspace_bytes, stream)


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


_plain_once = functools.lru_cache(maxsize=256)(_plain)


def _read(scoring, renormalize, scale, groups=1, top_groups=1, group_score="max"):
    """``_plain``, kept for options that are plain values themselves (a tensor is read at every call)."""
    kept = type(scale) is float and type(groups) is type(top_groups) is int and type(renormalize) is bool
    return (_plain_once if kept else _plain)(scoring, renormalize, scale, groups, top_groups, group_score)


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

    If logits requires a gradient, so do the weights; the picks have none.  Forward-mode
    tangents are refused.
    """
    _no_tangents(logits, bias)
    options = _read(scoring, renormalize, scale, groups, top_groups, group_score)
    if logits.requires_grad or (bias is not None and bias.requires_grad):
        import torch
        if torch.is_grad_enabled() and bias is not None and bias.requires_grad:
            raise ValueError("bias gets no gradient: detach it")
        if torch.is_grad_enabled():
            # the backward call's options are the plain numbers of this one: a tensor may have changed by then
            return _route_node().apply(logits, top_k, bias, options,
                                       {"scoring": scoring, "renormalize": bool(options[1]), "scale": options[2]})
    return _route(logits, top_k, bias, options)


@_on_stream
def route_experts_backward(logits, ids, grad_weights, *, scoring="softmax", renormalize=True, scale=1.0):
    """The gradient of ``sum(grad_weights * weights)`` with respect to
    ``logits``, [T, E] in its type, for ``ids`` and the options of the forward
    call.  It is outside torch's graph."""
    options = _read(scoring, renormalize, scale)
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


# ------------------------------------------------------- the experts' products

@functools.lru_cache(maxsize=1024)
def _experts_size(backward, sizes, in_offset, ld_in, out_offset, ld_out, code):
    st, n = experts_workspace_size(backward, *sizes, in_offset, ld_in, out_offset, ld_out, code)
    if st != OK:
        raise TgemmError(st, "tgemm_experts_workspace_size")
    return n


@functools.lru_cache(maxsize=1024)
def _saved_size(sizes, code):
    st, n = experts_saved_size(*sizes, code)
    if st != OK:
        raise TgemmError(st, "tgemm_experts_saved_size")
    return n


def _expert_rows(name, t, rows, cols):
    """Row pitch of the matrices [E, rows, cols] of one weight, which follow one another."""
    each, ld, step = t.stride()
    E = t.shape[0]
    if (cols > 1 and step != 1) or (rows > 1 and ld < cols):
        raise ValueError(f"{name} must have unit column stride and rows that do not overlap")
    if rows < 2:
        ld = each if E > 1 else cols
    if E > 1 and each != rows * ld:
        raise ValueError(f"{name}: each expert's rows must follow the last one's")
    if ld < cols:
        raise ValueError(f"{name} must have unit column stride and rows that do not overlap")
    return ld


def _experts(hidden, w_in, w_out, ids, weights, backward, workspace):
    """Checks what both calls share: (torch, device, (T, E, k, D, F), dtype code, matrices' arguments, ids, weights,
    workspace, its bytes)."""
    import torch
    if hidden.dim() != 2 or w_in.dim() != 3 or w_out.dim() != 3 or ids.dim() != 2:
        raise ValueError("hidden [T, D], w_in [E, 2 F, D], w_out [E, D, F] and ids [T, k] must have these dimensions")
    T, D = hidden.shape
    E, _, F = w_out.shape
    k = ids.shape[1]
    dtype = hidden.dtype
    code = {torch.bfloat16: BF16, torch.float16: F16}.get(dtype)
    if code is None:
        raise ValueError(f"unsupported dtype: {dtype} (bf16 or fp16)")
    if w_in.shape != (E, 2 * F, D) or w_out.shape != (E, D, F) or w_in.dtype != dtype or w_out.dtype != dtype:
        raise ValueError(f"w_in must be [E, 2 F, {D}] and w_out [E, {D}, F] {dtype}, got {tuple(w_in.shape)} "
                         f"{w_in.dtype} and {tuple(w_out.shape)} {w_out.dtype}")
    device = hidden.get_device()
    if device < 0 or w_in.get_device() != device or w_out.get_device() != device:
        raise ValueError("hidden, w_in and w_out must be on one CUDA device")
    shape = torch.Size((T, k))
    ids = _places("ids", ids, shape, torch.int64, device)
    weights = _places("weights", weights, shape, torch.float32, device)
    sizes = (T, E, k, D, F)
    ldx, ld_in, ld_out = _pitch("hidden", hidden, T, D), _expert_rows("w_in", w_in, 2 * F, D), \
        _expert_rows("w_out", w_out, D, F)
    p_in, p_out = w_in.data_ptr(), w_out.data_ptr()
    need = _experts_size(backward, sizes, p_in % 16, ld_in, p_out % 16, ld_out, code)
    workspace, need = _lent("workspace", workspace, need, device, hidden)
    return torch, device, sizes, code, (hidden.data_ptr(), ldx, p_in, ld_in, p_out, ld_out), ids, weights, workspace, need


def _lent(name, buffer, need, device, like):
    """A buffer of at least `need` bytes, and its size."""
    import torch
    if buffer is None:
        return torch.empty(need, dtype=torch.uint8, device=like.device), need
    if buffer.get_device() != device or buffer.dtype != torch.uint8 or not buffer.is_contiguous() or \
            buffer.numel() < need:
        raise ValueError(f"{name} must be a contiguous uint8 tensor of at least {need} bytes on the device of hidden")
    return buffer, buffer.numel()


@functools.cache
def _mlp_node():
    """The torch function that records experts' products whose operands require a gradient."""
    import torch

    class ExpertMLP(torch.autograd.Function):
        @staticmethod
        def forward(ctx, hidden, w_in, w_out, ids, weights, workspace):
            ctx.set_materialize_grads(False)
            out, saved = _mlp(hidden, w_in, w_out, ids, weights, True, workspace)
            ctx.save_for_backward(hidden, w_in, w_out, ids, weights, saved)
            ctx.mark_non_differentiable(saved)
            return out, saved

        @staticmethod
        @torch.autograd.function.once_differentiable
        def backward(ctx, grad, _):
            if grad is None:
                return (None,) * 6
            hidden, w_in, w_out, ids, weights, saved = ctx.saved_tensors
            want = ctx.needs_input_grad
            dx, dw_in, dw_out, dw = expert_mlp_backward(hidden, w_in, w_out, ids, weights, saved, grad,
                                                        want_hidden=want[0], want_in=want[1], want_out=want[2],
                                                        want_weights=want[4])
            return dx, dw_in, dw_out, None, dw, None

    return ExpertMLP


def _mlp(hidden, w_in, w_out, ids, weights, save, workspace):
    torch, device, sizes, code, matrices, ids, weights, workspace, need = \
        _experts(hidden, w_in, w_out, ids, weights, False, workspace)
    T, D = hidden.shape
    out = torch.empty((T, D), dtype=hidden.dtype, device=hidden.device)
    saved = torch.empty(_saved_size(sizes, code), dtype=torch.uint8, device=hidden.device) if save else None
    st = _guarded(torch, device, _lib.tgemm_experts_forward,
                  sizes + matrices + (ids.data_ptr(), weights.data_ptr(), code, None, out.data_ptr(), D,
                                      saved.data_ptr() if save else 0, saved.numel() if save else 0,
                                      workspace.data_ptr(), need, _current_stream(torch, device)))
    if st != OK:
        raise TgemmError(st, "tgemm_experts_forward")
    return out, saved


@_on_stream
def expert_mlp(hidden, w_in, w_out, ids, weights, *, save=False, workspace=None):
    """``out[t] = sum_j weights[t, j] * w_out[e] @ (silu(g) * u)`` with ``e =
    ids[t, j]`` and ``(g, u) = w_in[e] @ hidden[t]``: ``(out [T, D], saved)``.

    hidden [T, D], w_in [E, 2 F, D] (F gates, then F ups) and w_out [E, D, F] in
    bf16 or fp16, unit column stride, any row stride; ids [T, k] int64 (below 0:
    unused place) and weights [T, k] float32, as route_experts gives them.  A
    row without a used place gives 0, whatever hidden holds there.  h = silu(g) * u is
    rounded to the operands' type (fp16: beyond 65504 it is infinite), out once more.

    save=True keeps what expert_mlp_backward takes (a uint8 tensor: the rows'
    order, the rows in it, g and u in float32); otherwise saved is None.  If
    hidden, a weight or weights requires a gradient, so does out, torch's
    backward pass makes the backward call, and saved is kept in any case.
    Forward-mode tangents are refused.
    """
    _no_tangents(hidden, w_in, w_out, weights)
    if hidden.requires_grad or w_in.requires_grad or w_out.requires_grad or weights.requires_grad:
        import torch
        if torch.is_grad_enabled():
            return _mlp_node().apply(hidden, w_in, w_out, ids, weights, workspace)
    return _mlp(hidden, w_in, w_out, ids, weights, bool(save), workspace)


@_on_stream
def expert_mlp_backward(hidden, w_in, w_out, ids, weights, saved, grad_out, *, want_hidden=True, want_in=True,
                        want_out=True, want_weights=True, workspace=None):
    """Gradients ``(d_hidden, d_w_in, d_w_out, d_weights)`` of ``sum(grad_out *
    out)``: in the operands' type, d_weights in float32.  saved from the forward
    call with the same operands; grad_out [T, D] in their type, unit column stride.  An
    unwanted gradient is not computed (None), the others are the same bits.  What it
    returns is outside torch's graph."""
    torch, device, sizes, code, matrices, ids, weights, workspace, need = \
        _experts(hidden, w_in, w_out, ids, weights, True, workspace)
    T, E, k, D, F = sizes
    if saved is None:
        raise ValueError("saved is what expert_mlp(..., save=True) gives")
    saved, kept = _lent("saved", saved, _saved_size(sizes, code), device, hidden)
    if grad_out.shape != hidden.shape or grad_out.dtype != hidden.dtype or grad_out.get_device() != device:
        raise ValueError(f"grad_out must be [{T}, {D}] {hidden.dtype} on the device of hidden")
    if T and (grad_out.stride(1) != 1 and D > 1 or grad_out.stride(0) < D and T > 1):
        grad_out = grad_out.contiguous()

    def make(wanted, *shape, dtype=hidden.dtype):
        return torch.empty(shape, dtype=dtype, device=hidden.device) if wanted else None

    def at(t):
        return 0 if t is None else t.data_ptr()

    dx, dw_in, dw_out = make(want_hidden, T, D), make(want_in, E, 2 * F, D), make(want_out, E, D, F)
    dw = make(want_weights, T, k, dtype=torch.float32)
    st = _guarded(torch, device, _lib.tgemm_experts_backward,
                  sizes + matrices + (weights.data_ptr(), saved.data_ptr(), kept, grad_out.data_ptr(),
                                      _pitch("grad_out", grad_out, T, D), code, None, at(dx), D, at(dw_in), D, at(dw_out),
                                      F, at(dw), workspace.data_ptr(), need, _current_stream(torch, device)))
    if st != OK:
        raise TgemmError(st, "tgemm_experts_backward")
    return dx, dw_in, dw_out, dw
