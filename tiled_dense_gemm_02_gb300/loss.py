"""Vocabulary-head losses (``include/tgemm_loss.h``): the product of hidden
states with a head's weight, fused with the cross entropy or the distillation
loss that reads it, and its gradient.  The T x V logits are never written.

The first functions carry the names of the C ABI and only marshal arguments;
``linear_cross_entropy``, ``linear_distillation`` and their ``_backward`` take
torch tensors (torch supplies device memory and streams only).
"""
from __future__ import annotations

import ctypes
import functools
import math
from operator import index

from . import BF16, F16, F32, OK, TgemmError, library

DISTILL_MAX_K = 256  # TGEMM_DISTILL_MAX_K

LOSS_EXPORTS = ("tgemm_loss_workspace_size", "tgemm_xent_forward", "tgemm_xent_backward", "tgemm_distill_forward",
                "tgemm_distill_backward")


class LossOptions(ctypes.Structure):
    """struct tgemm_loss_options"""
    _fields_ = [("scale", ctypes.c_float), ("label_smoothing", ctypes.c_float), ("z_loss", ctypes.c_float),
                ("piece", ctypes.c_int), ("ignore_index", ctypes.c_int64), ("wait_timeout_us", ctypes.c_int),
                ("reserved", ctypes.c_int * 3)]


def _declare(lib):
    i64, vp, ip, sz = ctypes.c_int64, ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
    op = ctypes.POINTER(LossOptions)
    lib.tgemm_loss_workspace_size.argtypes = [ip, i64, i64, i64, i64, vp, i64, ip, op, ctypes.POINTER(sz)]
    lib.tgemm_xent_forward.argtypes = [i64, i64, i64, vp, i64, vp, i64, vp, ip, op, vp, vp, vp, sz, vp]
    lib.tgemm_xent_backward.argtypes = [i64, i64, i64, vp, i64, vp, i64, vp, vp, vp, ip, op, vp, i64, vp, i64, vp, sz,
                                        vp]
    lib.tgemm_distill_forward.argtypes = [i64, i64, i64, i64, vp, i64, vp, i64, vp, i64, vp, i64, ip, op, vp, vp, vp,
                                          sz, vp]
    lib.tgemm_distill_backward.argtypes = [i64, i64, i64, i64, vp, i64, vp, i64, vp, i64, vp, i64, vp, vp, ip, op, vp,
                                           i64, vp, i64, vp, sz, vp]
    for name in LOSS_EXPORTS:
        getattr(lib, name).restype = ip
    return lib


_lib = _declare(library())


def _opts(options):
    if options is None:
        return None
    if isinstance(options, LossOptions):
        return ctypes.byref(options)
    o = LossOptions(ignore_index=-100)
    for k, v in dict(options).items():
        setattr(o, k, v)
    return ctypes.byref(o)


def loss_workspace_size(backward, T, V, D, K, W, ldw, dtype, options=None):
    """tgemm_loss_workspace_size: (status, bytes); needs no GPU."""
    n = ctypes.c_size_t(0)
    st = _lib.tgemm_loss_workspace_size(int(backward), T, V, D, K, W, ldw, dtype, _opts(options), ctypes.byref(n))
    return st, n.value


def xent_forward(T, V, D, H, ldh, W, ldw, targets, dtype, loss, lse, options=None, workspace=0, workspace_bytes=0,
                 stream=0) -> int:
    """tgemm_xent_forward: device pointers as ints; returns the status."""
    return _lib.tgemm_xent_forward(T, V, D, H, ldh, W, ldw, targets, dtype, _opts(options), loss, lse, workspace,
                                   workspace_bytes, stream)


def xent_backward(T, V, D, H, ldh, W, ldw, targets, lse, grad, dtype, dH, lddh, dW, lddw, options=None, workspace=0,
                  workspace_bytes=0, stream=0) -> int:
    """tgemm_xent_backward: dH or dW may be 0 when it is not wanted."""
    return _lib.tgemm_xent_backward(T, V, D, H, ldh, W, ldw, targets, lse, grad, dtype, _opts(options), dH, lddh, dW,
                                    lddw, workspace, workspace_bytes, stream)


def distill_forward(T, V, D, K, H, ldh, W, ldw, ids, ld_ids, logits, ld_logits, dtype, loss, lse, options=None,
                    workspace=0, workspace_bytes=0, stream=0) -> int:
    """tgemm_distill_forward"""
    return _lib.tgemm_distill_forward(T, V, D, K, H, ldh, W, ldw, ids, ld_ids, logits, ld_logits, dtype,
                                      _opts(options), loss, lse, workspace, workspace_bytes, stream)


def distill_backward(T, V, D, K, H, ldh, W, ldw, ids, ld_ids, logits, ld_logits, lse, grad, dtype, dH, lddh, dW, lddw,
                     options=None, workspace=0, workspace_bytes=0, stream=0) -> int:
    """tgemm_distill_backward: dH or dW may be 0 when it is not wanted."""
    return _lib.tgemm_distill_backward(T, V, D, K, H, ldh, W, ldw, ids, ld_ids, logits, ld_logits, lse, grad, dtype,
                                       _opts(options), dH, lddh, dW, lddw, workspace, workspace_bytes, stream)


# ------------------------------------------------------------ torch helpers
# The checks below read each property of a tensor once, and what depends on
# plain numbers only (options, workspace sizes) is computed once per set of
# numbers: a call costs the host little more than its launches.

@functools.lru_cache(maxsize=256)
def _options(scale, label_smoothing, z_loss, piece, ignore_index):
    return ctypes.byref(LossOptions(scale=scale, label_smoothing=label_smoothing, z_loss=z_loss, piece=piece,
                                    ignore_index=ignore_index))


@functools.lru_cache(maxsize=1024)
def _size(backward, T, V, D, K, w_offset, ldw, code, options):
    n = ctypes.c_size_t(0)
    st = _lib.tgemm_loss_workspace_size(int(backward), T, V, D, K, w_offset, ldw, code, options, ctypes.byref(n))
    if st != OK:
        raise TgemmError(st, "tgemm_loss_workspace_size")
    return n.value


def _pitch(name, t, rows, cols):
    """Row pitch of a matrix with unit column stride and rows that do not overlap."""
    ld, step = t.stride()
    if rows < 2:
        ld = cols
    elif ld < cols:
        raise ValueError(f"{name} must have rows that do not overlap")
    if cols > 1 and step != 1 and rows:
        raise ValueError(f"{name} must have unit column stride")
    return ld or 1


def _vector(name, t, n, dtype, device):
    if t.dim() != 1 or t.shape[0] != n or t.dtype != dtype:
        raise ValueError(f"{name} must be a vector of {n} {dtype} values, got {tuple(t.shape)} {t.dtype}")
    if t.get_device() != device:
        raise ValueError(f"{name} must be on the device of hidden")
    return t if n < 2 or t.stride(0) == 1 else t.contiguous()


def _on_stream(function):
    """Adds ``stream`` (a cudaStream_t as int; default: the current stream): the
    whole call runs with that stream current, so its workspace, outputs and
    converted inputs belong to it."""

    @functools.wraps(function)
    def call(hidden, *args, stream=None, **kwargs):
        if stream is None:
            return function(hidden, *args, **kwargs)
        import torch
        other = torch.cuda.ExternalStream(stream, device=hidden.device) if stream else \
            torch.cuda.default_stream(hidden.device)
        with torch.cuda.stream(other):
            return function(hidden, *args, **kwargs)

    return call


def _head(hidden, weight, backward, K, options, workspace):
    """Checks what every call shares: (torch, device, (T, V, D), dtype code, matrices' arguments, options, workspace)."""
    import torch
    if hidden.dim() != 2 or weight.dim() != 2:
        raise ValueError("hidden [T, D] and weight [V, D] must be matrices")
    T, D = hidden.shape
    V, columns = weight.shape
    dtype = hidden.dtype
    if columns != D or weight.dtype != dtype:
        raise ValueError(f"weight must be [V, {D}] {dtype}, got {tuple(weight.shape)} {weight.dtype}")
    code = BF16 if dtype == torch.bfloat16 else F16 if dtype == torch.float16 else F32
    if code == F32 and dtype != torch.float32:
        raise ValueError(f"unsupported dtype: {dtype}")
    device = hidden.get_device()
    if device < 0 or weight.get_device() != device:
        raise ValueError("hidden and weight must be on one CUDA device")
    ldh, ldw = _pitch("hidden", hidden, T, D), _pitch("weight", weight, V, D)
    w = weight.data_ptr()
    options = _options(*options)
    need = _size(backward, T, V, D, K, w % 16, ldw, code, options)
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=hidden.device)
    elif workspace.get_device() != device or workspace.dtype != torch.uint8 or not workspace.is_contiguous() or \
            workspace.numel() < need:
        raise ValueError(f"workspace must be a contiguous uint8 tensor of at least {need} bytes on the device of hidden")
    else:
        need = workspace.numel()
    return torch, device, (T, V, D), code, (hidden.data_ptr(), ldh, w, ldw), options, workspace, need


def _current_stream(torch, device):
    """The current stream's handle; torch's own short way to it where there is one (1 us of a 20 us call)."""
    raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    return raw(device) if raw else torch.cuda.current_stream(device).cuda_stream


def _guarded(torch, device, function, args):
    """``function(*args)`` with ``device`` current: the library launches on the current device."""
    if torch.cuda.current_device() == device:
        return function(*args)
    with torch.cuda.device(device):
        return function(*args)


def _call(torch, device, function, args, workspace, need):
    st = _guarded(torch, device, function, args + (workspace.data_ptr(), need, _current_stream(torch, device)))
    if st != OK:
        raise TgemmError(st, function.__name__)


def _losses(torch, T, device):
    # two allocations cost less than two views of one
    return torch.empty(T, dtype=torch.float32, device=device), torch.empty(T, dtype=torch.float32, device=device)


def _gradients(torch, hidden, sizes, want_hidden, want_weight):
    """Outputs in the operands' type, with their pointers and pitches (0 when not wanted)."""
    T, V, D = sizes
    dh = torch.empty((T, D), dtype=hidden.dtype, device=hidden.device) if want_hidden else None
    dw = torch.empty((V, D), dtype=hidden.dtype, device=hidden.device) if want_weight else None
    return dh, dw, (dh.data_ptr() if want_hidden else 0, D, dw.data_ptr() if want_weight else 0, D)


def _factor(name, value, invert=False):
    """The logits' factor from ``value`` or, inverted, its reciprocal.  The library holds it in float32, where 0 stands
    for the default: what rounds to 0 or to infinity there is refused."""
    value = float(value)
    factor = ctypes.c_float(1.0 / value if invert and value else value).value
    if not (value > 0.0 and 0.0 < factor < math.inf):
        raise ValueError(f"{name} must be positive{', its reciprocal' if invert else ''} within float32's range, "
                         f"got {value}")
    return factor


def _plain(scale, label_smoothing, z_loss, piece, ignore_index):
    """The options as plain numbers, read now: the cache of ``_options`` goes by value, a tensor's key is its identity."""
    return _factor("scale", scale), float(label_smoothing), float(z_loss), index(piece), index(ignore_index)


@functools.cache
def _graph_node():
    """The torch function that records a loss: what a loss of tensors that require a gradient goes through."""
    import torch

    class HeadLoss(torch.autograd.Function):
        @staticmethod
        def forward(ctx, hidden, weight, forward, backward, lists, more, workspace):
            ctx.set_materialize_grads(False)
            loss, lse = forward(hidden, weight, *lists, workspace=workspace, **more)
            ctx.save_for_backward(hidden, weight, lse, *lists)
            ctx.call = backward, more
            return loss, lse

        @staticmethod
        @torch.autograd.function.once_differentiable
        def backward(ctx, grad_loss, grad_lse):
            if grad_lse is not None:
                raise RuntimeError("lse has no gradient of its own (z_loss weighs its square): detach it")
            d_hidden = d_weight = None
            if grad_loss is not None:
                hidden, weight, lse, *lists = ctx.saved_tensors
                backward, more = ctx.call
                d_hidden, d_weight = backward(hidden, weight, *lists, lse, grad_loss, want_hidden=ctx.needs_input_grad[0],
                                              want_weight=ctx.needs_input_grad[1], **more)
            return d_hidden, d_weight, None, None, None, None, None

    return HeadLoss


def _no_tangents(*tensors):
    """Refuses forward-mode duals: there is no forward-mode gradient, and the library would read past a tangent."""
    from torch.autograd import forward_ad
    if getattr(forward_ad, "_current_level", 0) < 0:  # not in forward mode
        return
    for t in tensors:
        if t is not None and forward_ad.unpack_dual(t).tangent is not None:
            raise RuntimeError("there is no forward-mode gradient: unpack the dual tensor")


def _recorded(hidden, weight):
    """Whether a loss of these tensors belongs to torch's graph."""
    if not (hidden.requires_grad or weight.requires_grad):
        return False
    import torch
    return torch.is_grad_enabled()


@_on_stream
def linear_cross_entropy(hidden, weight, targets, *, ignore_index=-100, scale=1.0, label_smoothing=0.0, z_loss=0.0,
                         piece=0, workspace=None):
    """Cross entropy of ``scale * hidden @ weight.T`` against ``targets``, one
    float32 loss per row, without the logits: ``(loss [T], lse [T])``.

    hidden [T, D], weight [V, D] (bf16, fp16 or fp32, unit column stride, any
    row stride), targets [T] int64.  Rows whose target is ``ignore_index`` get
    loss and lse 0.  ``lse`` is the log of the sum of exponentials, which the
    backward call takes.  Reduce as you like: ``loss.sum() / n``.

    If hidden or weight requires a gradient, so does ``loss``, and torch's
    backward pass makes the backward call; ``lse`` has no gradient of its own.
    Forward-mode tangents are refused.
    """
    _no_tangents(hidden, weight)
    options = _plain(scale, label_smoothing, z_loss, piece, ignore_index)
    if _recorded(hidden, weight):
        more = dict(zip(("scale", "label_smoothing", "z_loss", "piece", "ignore_index"), options))
        return _graph_node().apply(hidden, weight, linear_cross_entropy, linear_cross_entropy_backward, (targets,),
                                   more, workspace)
    torch, device, sizes, code, matrices, options, workspace, need = _head(hidden, weight, False, 0, options, workspace)
    targets = _vector("targets", targets, sizes[0], torch.int64, device)
    loss, lse = _losses(torch, sizes[0], hidden.device)
    _call(torch, device, _lib.tgemm_xent_forward, sizes + matrices + (targets.data_ptr(), code, options,
                                                                      loss.data_ptr(), lse.data_ptr()),
          workspace, need)
    return loss, lse


@_on_stream
def linear_cross_entropy_backward(hidden, weight, targets, lse, grad_loss, *, ignore_index=-100, scale=1.0,
                                  label_smoothing=0.0, z_loss=0.0, piece=0, want_hidden=True, want_weight=True,
                                  workspace=None):
    """Gradients ``(d_hidden, d_weight)`` of ``sum(grad_loss * loss)`` in the
    operands' type; ``lse`` from the forward call with the same options,
    grad_loss [T] float32.  An unwanted gradient is not computed (None).  What
    it returns is outside torch's graph."""
    options = _plain(scale, label_smoothing, z_loss, piece, ignore_index)
    torch, device, sizes, code, matrices, options, workspace, need = _head(hidden, weight, True, 0, options, workspace)
    targets = _vector("targets", targets, sizes[0], torch.int64, device)
    lse = _vector("lse", lse, sizes[0], torch.float32, device)
    grad_loss = _vector("grad_loss", grad_loss, sizes[0], torch.float32, device)
    dh, dw, out = _gradients(torch, hidden, sizes, want_hidden, want_weight)
    _call(torch, device, _lib.tgemm_xent_backward,
          sizes + matrices + (targets.data_ptr(), lse.data_ptr(), grad_loss.data_ptr(), code, options) + out,
          workspace, need)
    return dh, dw


def _teacher(hidden, weight, backward, ids, logits, temperature, piece, workspace):
    """What _head gives, the teacher's logits in float32, and the lists' arguments."""
    if ids.dim() != 2 or logits.shape != ids.shape:
        raise ValueError("teacher_ids and teacher_logits must be matrices of one shape [T, K]")
    rows, K = ids.shape
    if K < 1:
        raise ValueError("the teacher's lists must have at least one place")
    head = _head(hidden, weight, backward, K, (_factor("temperature", temperature, True), 0.0, 0.0, index(piece), 0),
                 workspace)
    torch, device, sizes = head[:3]
    if rows != sizes[0] or ids.dtype != torch.int64:
        raise ValueError(f"teacher_ids must be [{sizes[0]}, K] int64, got {tuple(ids.shape)} {ids.dtype}")
    if ids.get_device() != device or logits.get_device() != device:
        raise ValueError("teacher_ids and teacher_logits must be on the device of hidden")
    if logits.dtype != torch.float32:
        logits = logits.float()
    return head, logits, (ids.data_ptr(), _pitch("teacher_ids", ids, rows, K), logits.data_ptr(),
                          _pitch("teacher_logits", logits, rows, K))


@_on_stream
def linear_distillation(hidden, weight, teacher_ids, teacher_logits, *, temperature=1.0, piece=0, workspace=None):
    """Divergence of the student ``hidden @ weight.T / temperature`` from the
    teacher's renormalised top logits, one float32 loss per row, without the
    student's logits: ``(loss [T], lse [T])``.

    teacher_ids [T, K] int64 (below 0: unused place), teacher_logits [T, K] in
    any float type, K up to 256.  A row without a used place gets loss and lse
    0.  The losses are not multiplied by temperature squared.

    Gradients of hidden and weight through torch as in linear_cross_entropy;
    teacher_logits have none and must not require one.  Forward-mode tangents are refused.
    """
    _no_tangents(hidden, weight, teacher_logits)
    if teacher_logits.requires_grad:
        import torch
        if torch.is_grad_enabled():
            raise ValueError("teacher_logits get no gradient: detach them")
    if _recorded(hidden, weight):
        return _graph_node().apply(hidden, weight, linear_distillation, linear_distillation_backward,
                                   (teacher_ids, teacher_logits),
                                   {"temperature": float(temperature), "piece": index(piece)}, workspace)
    head, logits, lists = _teacher(hidden, weight, False, teacher_ids, teacher_logits, temperature, piece, workspace)
    torch, device, sizes, code, matrices, options, workspace, need = head
    loss, lse = _losses(torch, sizes[0], hidden.device)
    _call(torch, device, _lib.tgemm_distill_forward,
          (*sizes, logits.shape[1], *matrices, *lists, code, options, loss.data_ptr(), lse.data_ptr()), workspace, need)
    return loss, lse


@_on_stream
def linear_distillation_backward(hidden, weight, teacher_ids, teacher_logits, lse, grad_loss, *, temperature=1.0,
                                 piece=0, want_hidden=True, want_weight=True, workspace=None):
    """Gradients ``(d_hidden, d_weight)`` of ``sum(grad_loss * loss)``; lse,
    grad_loss and unwanted gradients as in linear_cross_entropy_backward."""
    head, logits, lists = _teacher(hidden, weight, True, teacher_ids, teacher_logits, temperature, piece, workspace)
    torch, device, sizes, code, matrices, options, workspace, need = head
    lse = _vector("lse", lse, sizes[0], torch.float32, device)
    grad_loss = _vector("grad_loss", grad_loss, sizes[0], torch.float32, device)
    dh, dw, out = _gradients(torch, hidden, sizes, want_hidden, want_weight)
    _call(torch, device, _lib.tgemm_distill_backward,
          (*sizes, logits.shape[1], *matrices, *lists, lse.data_ptr(), grad_loss.data_ptr(), code, options, *out),
          workspace, need)
    return dh, dw
