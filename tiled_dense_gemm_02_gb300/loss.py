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

def _ld(t):
    return max(t.stride(0), t.shape[1], 1) if t.shape[0] > 1 else max(t.shape[1], 1)


def _matrix(name, t, rows=None, cols=None, dtype=None):
    if t.dim() != 2 or (rows is not None and t.shape[0] != rows) or (cols is not None and t.shape[1] != cols):
        raise ValueError(f"{name} must be a matrix of shape [{'T' if rows is None else rows}, "
                         f"{'D' if cols is None else cols}], got {tuple(t.shape)}")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape[0] > 1 and t.shape[1] > 0 and t.stride(0) < t.shape[1]:
        raise ValueError(f"{name} must have rows that do not overlap")
    if t.numel() and t.shape[1] > 1 and t.stride(1) != 1:
        raise ValueError(f"{name} must have unit column stride")


def _vector(name, t, n, dtype):
    if t.dim() != 1 or t.shape[0] != n or t.dtype != dtype:
        raise ValueError(f"{name} must be a vector of {n} {dtype} values, got {tuple(t.shape)} {t.dtype}")
    return t if n < 2 or t.stride(0) == 1 else t.contiguous()


def _on_stream(function):
    """Adds ``stream`` (a cudaStream_t as int; default: the current stream): the
    whole call runs with that stream current, so its workspace, outputs and
    converted inputs belong to it."""

    @functools.wraps(function)
    def call(hidden, *args, stream=None, **kwargs):
        import torch
        if stream is None:
            return function(hidden, *args, **kwargs)
        other = torch.cuda.ExternalStream(stream, device=hidden.device) if stream else \
            torch.cuda.default_stream(hidden.device)
        with torch.cuda.stream(other):
            return function(hidden, *args, **kwargs)

    return call


class _Head:
    """The arguments every call shares, checked."""

    def __init__(self, hidden, weight, options, workspace, backward, K):
        import torch
        self.torch = torch
        _matrix("hidden", hidden)
        _matrix("weight", weight, cols=hidden.shape[1], dtype=hidden.dtype)
        codes = {torch.float32: F32, torch.float16: F16, torch.bfloat16: BF16}
        if hidden.dtype not in codes:
            raise ValueError(f"unsupported dtype: {hidden.dtype}")
        for name, t in (("hidden", hidden), ("weight", weight)):
            if not t.is_cuda or t.device != hidden.device:
                raise ValueError(f"{name} must be on one CUDA device")
        self.hidden, self.weight, self.dev = hidden, weight, hidden.device
        self.T, self.D, self.V = hidden.shape[0], hidden.shape[1], weight.shape[0]
        self.code = codes[hidden.dtype]
        self.ldh, self.ldw = _ld(hidden), _ld(weight)
        self.options = _opts(options)
        self.stream = torch.cuda.current_stream(self.dev).cuda_stream
        n = ctypes.c_size_t(0)
        self.check(_lib.tgemm_loss_workspace_size(int(backward), self.T, self.V, self.D, K, weight.data_ptr(),
                                                  self.ldw, self.code, self.options, ctypes.byref(n)),
                   "tgemm_loss_workspace_size")
        if workspace is None:
            workspace = torch.empty(n.value, dtype=torch.uint8, device=self.dev)
        elif workspace.device != self.dev or workspace.dtype != torch.uint8 or not workspace.is_contiguous() or workspace.numel() < n.value:
            raise ValueError(f"workspace must be a contiguous uint8 tensor of at least {n.value} bytes on {self.dev}")
        self.workspace = workspace

    def on_device(self, *named):
        for name, t in named:
            if t.device != self.dev:
                raise ValueError(f"{name} must be on {self.dev}")

    @staticmethod
    def check(status, where):
        if status != OK:
            raise TgemmError(status, where)

    def call(self, function, *args):
        with self.torch.cuda.device(self.dev):
            st = function(*args, self.workspace.data_ptr(), self.workspace.numel(), self.stream)
        self.check(st, function.__name__)

    def head_args(self):
        return self.hidden.data_ptr(), self.ldh, self.weight.data_ptr(), self.ldw

    def losses(self):
        both = self.torch.empty((2, self.T), dtype=self.torch.float32, device=self.dev)
        return both[0], both[1]

    def gradients(self, want_hidden, want_weight):
        """Outputs in the operands' type; their pointers and pitches (0 when not wanted)."""
        torch = self.torch
        dh = torch.empty((self.T, self.D), dtype=self.hidden.dtype, device=self.dev) if want_hidden else None
        dw = torch.empty((self.V, self.D), dtype=self.weight.dtype, device=self.dev) if want_weight else None
        args = (dh.data_ptr() if want_hidden else 0, max(self.D, 1), dw.data_ptr() if want_weight else 0,
                max(self.D, 1))
        return dh, dw, args


def _xent_options(ignore_index, scale, label_smoothing, z_loss, piece):
    return LossOptions(scale=scale, label_smoothing=label_smoothing, z_loss=z_loss, piece=piece,
                       ignore_index=ignore_index)


def _positive(name, value):
    if not value > 0:
        raise ValueError(f"{name} must be positive, got {value}")
    return value


@_on_stream
def linear_cross_entropy(hidden, weight, targets, *, ignore_index=-100, scale=1.0, label_smoothing=0.0, z_loss=0.0,
                         piece=0, workspace=None):
    """Cross entropy of ``scale * hidden @ weight.T`` against ``targets``, one
    float32 loss per row, without the logits: ``(loss [T], lse [T])``.

    hidden [T, D], weight [V, D] (bf16, fp16 or fp32, unit column stride, any
    row stride), targets [T] int64.  Rows whose target is ``ignore_index`` get
    loss and lse 0.  ``lse`` is the log of the sum of exponentials, which the
    backward call takes.  Reduce as you like: ``loss.sum() / n``.
    """
    h = _Head(hidden, weight, _xent_options(ignore_index, _positive("scale", scale), label_smoothing, z_loss, piece),
              workspace, False, 0)
    targets = _vector("targets", targets, h.T, h.torch.int64)
    h.on_device(("targets", targets))
    loss, lse = h.losses()
    h.call(_lib.tgemm_xent_forward, h.T, h.V, h.D, *h.head_args(), targets.data_ptr(), h.code, h.options,
           loss.data_ptr(), lse.data_ptr())
    return loss, lse


@_on_stream
def linear_cross_entropy_backward(hidden, weight, targets, lse, grad_loss, *, ignore_index=-100, scale=1.0,
                                  label_smoothing=0.0, z_loss=0.0, piece=0, want_hidden=True, want_weight=True,
                                  workspace=None):
    """Gradients ``(d_hidden, d_weight)`` of ``sum(grad_loss * loss)`` in the
    operands' type; ``lse`` from the forward call with the same options,
    grad_loss [T] float32.  An unwanted gradient is not computed (None)."""
    h = _Head(hidden, weight, _xent_options(ignore_index, _positive("scale", scale), label_smoothing, z_loss, piece),
              workspace, True, 0)
    f32 = h.torch.float32
    targets = _vector("targets", targets, h.T, h.torch.int64)
    lse, grad_loss = _vector("lse", lse, h.T, f32), _vector("grad_loss", grad_loss, h.T, f32)
    h.on_device(("targets", targets), ("lse", lse), ("grad_loss", grad_loss))
    dh, dw, out = h.gradients(want_hidden, want_weight)
    h.call(_lib.tgemm_xent_backward, h.T, h.V, h.D, *h.head_args(), targets.data_ptr(), lse.data_ptr(),
           grad_loss.data_ptr(), h.code, h.options, *out)
    return dh, dw


def _teacher(h, ids, logits):
    torch = h.torch
    _matrix("teacher_ids", ids, rows=h.T, dtype=torch.int64)
    logits = logits.float()
    _matrix("teacher_logits", logits, rows=h.T, cols=ids.shape[1])
    h.on_device(("teacher_ids", ids), ("teacher_logits", logits))
    return logits, (ids.data_ptr(), _ld(ids), logits.data_ptr(), _ld(logits))


@_on_stream
def linear_distillation(hidden, weight, teacher_ids, teacher_logits, *, temperature=1.0, piece=0, workspace=None):
    """Divergence of the student ``hidden @ weight.T / temperature`` from the
    teacher's renormalised top logits, one float32 loss per row, without the
    student's logits: ``(loss [T], lse [T])``.

    teacher_ids [T, K] int64 (below 0: unused place), teacher_logits [T, K] in
    any float type, K up to 256.  A row without a used place gets loss and lse
    0.  The losses are not multiplied by temperature squared.
    """
    h = _Head(hidden, weight, LossOptions(scale=1.0 / _positive("temperature", temperature), piece=piece), workspace,
              False, teacher_ids.shape[-1])
    logits, lists = _teacher(h, teacher_ids, teacher_logits)
    loss, lse = h.losses()
    h.call(_lib.tgemm_distill_forward, h.T, h.V, h.D, teacher_ids.shape[1], *h.head_args(), *lists, h.code, h.options,
           loss.data_ptr(), lse.data_ptr())
    return loss, lse


@_on_stream
def linear_distillation_backward(hidden, weight, teacher_ids, teacher_logits, lse, grad_loss, *, temperature=1.0,
                                 piece=0, want_hidden=True, want_weight=True, workspace=None):
    """Gradients ``(d_hidden, d_weight)`` of ``sum(grad_loss * loss)``; lse,
    grad_loss and unwanted gradients as in linear_cross_entropy_backward."""
    h = _Head(hidden, weight, LossOptions(scale=1.0 / _positive("temperature", temperature), piece=piece), workspace,
              True, teacher_ids.shape[-1])
    f32 = h.torch.float32
    logits, lists = _teacher(h, teacher_ids, teacher_logits)
    lse, grad_loss = _vector("lse", lse, h.T, f32), _vector("grad_loss", grad_loss, h.T, f32)
    h.on_device(("lse", lse), ("grad_loss", grad_loss))
    dh, dw, out = h.gradients(want_hidden, want_weight)
    h.call(_lib.tgemm_distill_backward, h.T, h.V, h.D, teacher_ids.shape[1], *h.head_args(), *lists, lse.data_ptr(),
           grad_loss.data_ptr(), h.code, h.options, *out)
    return dh, dw
