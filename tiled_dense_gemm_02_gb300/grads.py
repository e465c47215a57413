"""The norm over all gradients of a training step, and their clipping
(``include/tgemm_grads.h``), in a few launches however many tensors there are.

``grad_norm`` and ``grad_clip`` carry the names of the C ABI and only marshal
arguments; ``gradient_norm`` and ``clip_gradients`` take torch tensors (torch
supplies device memory and streams only).
"""
from __future__ import annotations

import ctypes
from array import array
from operator import attrgetter, index

from . import BF16, F16, F32, OK, TgemmError, library
from .loss import _current_stream, _guarded

GRAD_MAX_TENSORS = 1048576  # TGEMM_GRAD_MAX_TENSORS

GRAD_EXPORTS = ("tgemm_grad_workspace_size", "tgemm_grad_norm", "tgemm_grad_clip")


def _declare(lib):
    i64, vp, sz = ctypes.c_int64, ctypes.c_void_p, ctypes.c_size_t
    lib.tgemm_grad_workspace_size.argtypes = [i64, ctypes.POINTER(sz)]
    lib.tgemm_grad_norm.argtypes = [i64, vp, vp, vp, vp, vp, sz, vp]
    lib.tgemm_grad_clip.argtypes = [i64, vp, vp, vp, vp, ctypes.c_float, vp, vp, sz, vp]
    for name in GRAD_EXPORTS:
        getattr(lib, name).restype = ctypes.c_int
    return lib


_lib = _declare(library())


def grad_workspace_size(n):
    """tgemm_grad_workspace_size: (status, bytes); needs no GPU."""
    size = ctypes.c_size_t(0)
    st = _lib.tgemm_grad_workspace_size(n, ctypes.byref(size))
    return st, size.value


def _list(kind, values):
    """A host array of plain integers and its address (None for no list)."""
    if values is None:
        return None, None
    a = array(kind, values)
    return a, a.buffer_info()[0] if len(a) else None


def grad_norm(grads, counts, dtypes, norm, workspace=0, workspace_bytes=0, stream=0) -> int:
    """tgemm_grad_norm: lists of device pointers, element counts and dtype codes; returns the status."""
    (g, pg), (c, pc), (d, pd) = _list("Q", grads), _list("q", counts), _list("i", dtypes)
    return _lib.tgemm_grad_norm(len(g), pg, pc, pd, norm, workspace, workspace_bytes, stream)


def grad_clip(grads, counts, dtypes, outputs, max_norm, norm, workspace=0, workspace_bytes=0, stream=0) -> int:
    """tgemm_grad_clip: outputs is a list of device pointers, or None (in place)."""
    (g, pg), (c, pc), (d, pd), (o, po) = _list("Q", grads), _list("q", counts), _list("i", dtypes), _list("Q", outputs)
    return _lib.tgemm_grad_clip(len(g), pg, pc, pd, po, max_norm, norm, workspace, workspace_bytes, stream)


def _dense(t):
    """Whether the elements fill one range of memory without gaps or repeats."""
    if t.is_contiguous():
        return True
    step = 1
    for size, stride in sorted(zip(t.shape, t.stride()), key=lambda d: (d[1], d[0])):
        if size == 1:
            continue
        if stride != step:
            return False
        step *= size
    return True


def _tensors(name, tensors):
    """(device, pointers, counts, dtype codes, whether all are contiguous) of dense tensors on one CUDA device.  One pass
    per property, without a line of Python per tensor: a call may list thousands."""
    import torch
    codes, tensor = {torch.float32: F32, torch.float16: F16, torch.bfloat16: BF16}, torch.Tensor
    kinds = list(map(codes.get, map(attrgetter("dtype"), tensors)))
    if None in kinds:
        raise ValueError(f"{name}: unsupported dtype {tensors[kinds.index(None)].dtype}")
    devices = set(map(tensor.get_device, tensors))
    if len(devices) != 1 or -1 in devices:
        raise ValueError(f"{name} must be on one CUDA device")
    contiguous = all(map(tensor.is_contiguous, tensors))
    if not contiguous and not all(map(_dense, tensors)):
        raise ValueError(f"{name} must be dense: a view with gaps or repeats has no elements of its own")
    return devices.pop(), list(map(tensor.data_ptr, tensors)), list(map(tensor.numel, tensors)), kinds, contiguous


def _run(tensors, outputs, max_norm, workspace, stream):
    import torch
    tensors = list(tensors)
    if not tensors:
        raise ValueError("gradients must list at least one tensor")
    device, pointers, counts, kinds, contiguous = _tensors("gradients", tensors)
    places = None
    if outputs is not None:
        outputs = list(outputs)
        if len(outputs) != len(tensors):
            raise ValueError(f"outputs must list {len(tensors)} tensors, got {len(outputs)}")
        other, places, sizes, types, filled = _tensors("outputs", outputs)
        if other != device or sizes != counts or types != kinds:
            raise ValueError("outputs must have the gradients' sizes, dtypes and device")
        if not (contiguous and filled) and \
                not all([o.stride() == t.stride() and o.shape == t.shape for o, t in zip(outputs, tensors)]):
            raise ValueError("outputs must have the gradients' order of elements: shapes and strides")
    st, need = grad_workspace_size(len(tensors))
    if st != OK:
        raise TgemmError(st, "tgemm_grad_workspace_size")
    where = tensors[0].device
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=where)
    elif workspace.get_device() != device or workspace.dtype != torch.uint8 or not workspace.is_contiguous() or \
            workspace.numel() < need:
        raise ValueError(f"workspace must be a contiguous uint8 tensor of at least {need} bytes on the gradients' device")
    norm = torch.empty((), dtype=torch.float32, device=where)
    more = (norm.data_ptr(), workspace.data_ptr(), workspace.numel(), _current_stream(torch, device))
    if max_norm is None:
        st = _guarded(torch, device, grad_norm, (pointers, counts, kinds) + more)
    else:
        st = _guarded(torch, device, grad_clip, (pointers, counts, kinds, places, max_norm) + more)
        if st == OK:  # torch's graph is told what was written past it
            torch.autograd.graph.increment_version(tensors if outputs is None else outputs)
    if st != OK:
        raise TgemmError(st, "tgemm_grad_norm" if max_norm is None else "tgemm_grad_clip")
    return norm


def _with_stream(tensors, stream, call):
    """``call()`` with ``stream`` (a cudaStream_t as int; None: the current one) current."""
    if stream is None:
        return call()
    import torch
    device = tensors[0].device
    other = torch.cuda.ExternalStream(index(stream), device=device) if stream else torch.cuda.default_stream(device)
    with torch.cuda.stream(other):
        return call()


def gradient_norm(gradients, *, workspace=None, stream=None):
    """The square root of the sum of all elements' squares over ``gradients`` (a
    list of dense tensors: bf16, fp16, fp32, mixed), as a float32 tensor of no
    dimension.  Sums are held in 64 bits, so neither length nor the size of
    the values overflows them."""
    gradients = list(gradients)
    return _with_stream(gradients, stream, lambda: _run(gradients, None, None, workspace, stream))


def clip_gradients(gradients, max_norm, *, outputs=None, workspace=None, stream=None):
    """Scales ``gradients`` by ``max_norm / norm`` where their norm over all
    tensors is above ``max_norm``, in place or into ``outputs`` (tensors of the
    same sizes and order of elements; where nothing is scaled they get copies), and
    returns the norm before it, as ``gradient_norm`` does.  Outputs that lie like their
    gradients modulo 16 bytes are written three times as fast.

    The host does not wait.  A norm that is infinite or NaN scales nothing: the
    caller looks at it and skips the step.  In place, a tensor may be listed
    only once.  Neither the norm nor outputs are part of torch's graph, which does notice
    that the tensors were written.
    """
    max_norm = float(max_norm)
    if not max_norm >= 0.0:
        raise ValueError(f"max_norm must not be negative, got {max_norm}")
    gradients = list(gradients)
    return _with_stream(gradients, stream, lambda: _run(gradients, outputs, max_norm, workspace, stream))
