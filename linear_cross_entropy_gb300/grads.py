"""The global norm of many gradients and clipping by it, on the library's CUDA
kernels: a launch covers up to 1000 tensors of any sizes and types, and nothing
waits for the GPU.

    loss.backward()
    norm = clip_grad_norm_(model.parameters(), 1.0)  # 0-d fp32, before clipping

cce_clip_grads writes the clipped gradients in place or into other tensors
(say, the 32-bit buffers of an optimiser).  Calls run on the current stream of
the gradients' device and can be captured into a CUDA graph.
"""
from __future__ import annotations

import array
import ctypes
import math

import torch

from . import _lib
from .norm import TYPES, _current_device, _raw_stream

_l = _lib.load()
_grad_norm, _clip_grads, _workspace_bytes = _l.cce_grad_norm, _l.cce_clip_grads, _l.cce_grad_norm_workspace_bytes

CLIP_EPS = 1e-6  # added to the norm before the division


def grad_norm_workspace_bytes(n_dense, n_strided=0) -> int:
    return int(_workspace_bytes(n_dense, n_strided))


def _norm_code(norm_type):
    norm_type = float(norm_type)
    if norm_type == 2.0:
        return 2
    if norm_type == math.inf:
        return 0
    raise ValueError(f"norm_type must be 2 or infinity, got {norm_type}")


def _dims(g, o):
    """Dimensions of (size, stride of g, stride of o), outermost first, without
    those of size one and merged where both tensors' elements continue."""
    dims = []
    order = sorted(range(g.dim()), key=lambda d: (-o.stride(d), -g.stride(d)))
    for d in order:
        n, gs, os_ = g.shape[d], g.stride(d), o.stride(d)
        if n == 1:
            continue
        if dims and dims[-1][1] == n * gs and dims[-1][2] == n * os_:
            dims[-1] = (dims[-1][0] * n, gs, os_)
        else:
            dims.append((n, gs, os_))
    return dims


def _strided_row(g, o, written, dense, strided):
    """Appends a tensor that is not contiguous: to `dense` when g and o are one
    block in the same order all the same, else to `strided`."""
    dims = _dims(g, o)
    if written and any(os_ == 0 for _, _, os_ in dims):
        raise ValueError("an expanded tensor cannot be written: several of its elements share memory")
    code = TYPES[g.dtype] + (TYPES[o.dtype] << 8)
    if not dims or (len(dims) == 1 and dims[0][1] == 1 and dims[0][2] == 1):
        dense += (g.data_ptr(), o.data_ptr(), g.numel(), code)
        return
    if len(dims) > 4:
        raise ValueError(f"a tensor of shape {tuple(g.shape)} and strides {g.stride()} has more than 4 dimensions "
                         "that do not continue each other: make it contiguous")
    dims = [(1, 0, 0)] * (4 - len(dims)) + dims
    strided.append(_lib.Strided(g.data_ptr(), o.data_ptr(), TYPES[g.dtype], TYPES[o.dtype],
                                *((ctypes.c_int64 * 4)(*col) for col in zip(*dims))))


def _check(t, dev, what):
    if not isinstance(t, torch.Tensor) or t.layout != torch.strided:
        raise ValueError(f"{what} must be dense tensors")
    if not t.is_cuda:
        raise ValueError(f"{what} must be CUDA tensors (no CPU path)")
    if t.dtype not in TYPES:
        raise ValueError(f"{what} must be bfloat16, float16 or float32, got {t.dtype}")
    if t.device != dev:
        raise ValueError(f"{what} must be on one device, got {dev} and {t.device}")


def _tables(grads, outs, dev):
    """The library's tables of the tensors: (array of dense rows, list of strided ones)."""
    dense, strided, index, types = [], [], dev.index, TYPES
    try:
        if outs is None:
            outs = grads
            written = False
        else:
            written = True
        for g, o in zip(grads, outs):
            gt = types.get(g.dtype)
            if gt is None or g.get_device() != index:
                _check(g, dev, "gradients")
            if o is g:
                if g.is_contiguous():
                    at = g.data_ptr()
                    dense += (at, at, g.numel(), gt * 257)
                    continue
            else:
                ot = types.get(o.dtype)
                if ot is None or o.get_device() != index:
                    _check(o, dev, "out")
                if o.shape != g.shape:
                    raise ValueError(f"out must have the shapes of the gradients: {tuple(o.shape)} for "
                                     f"{tuple(g.shape)}")
                if g.is_contiguous() and o.is_contiguous():
                    dense += (g.data_ptr(), o.data_ptr(), g.numel(), gt + (ot << 8))
                    continue
            _check(g, dev, "gradients")
            _check(o, dev, "out")
            if g.numel():
                _strided_row(g, o, written, dense, strided)
    except (RuntimeError, AttributeError):  # what is no dense tensor has no such methods
        for t in (*grads, *outs):
            _check(t, dev, "gradients and out")
        raise
    return array.array("q", dense), strided


def _call(grads, outs, norm_type, max_norm, eps, stream):
    dev = grads[0].device
    if stream is not None:
        with torch.cuda.stream(stream):
            return _call(grads, outs, norm_type, max_norm, eps, None)
    if not grads[0].is_cuda:
        _check(grads[0], dev, "gradients")
    if dev.index != _current_device():
        with torch.cuda.device(dev):
            return _call(grads, outs, norm_type, max_norm, eps, None)
    dense, strided = _tables(grads, outs, dev)
    rows = len(dense) // 4
    norm = torch.empty((), dtype=torch.float32, device=dev)
    need = _workspace_bytes(rows, len(strided))
    ws = torch.empty(need, dtype=torch.uint8, device=dev)
    table = (_lib.Strided * len(strided))(*strided) if strided else None
    args = (dense.buffer_info()[0] if rows else 0, rows, ctypes.addressof(table) if strided else 0, len(strided),
            norm_type)
    if outs is None:
        st = _grad_norm(*args, norm.data_ptr(), ws.data_ptr(), need, _raw_stream(dev.index))
        _lib.check(st, "cce_grad_norm")
    else:
        st = _clip_grads(*args, max_norm, eps, norm.data_ptr(), ws.data_ptr(), need, _raw_stream(dev.index))
        _lib.check(st, "cce_clip_grads")
        # autograd learns that these were written
        torch.autograd.graph.increment_version([o for o in outs if not o.is_inference()])
    return norm


def cce_grad_norm(grads, norm_type=2.0, *, stream=None):
    """The norm (0-d fp32) over all values of the tensors together: 2 or
    infinity.  Without tensors it is a 0 on the CPU."""
    grads = list(grads)
    code = _norm_code(norm_type)
    if not grads:
        return torch.zeros(())
    return _call(grads, None, code, 0.0, 0.0, stream)


def cce_clip_grads(grads, max_norm, norm_type=2.0, *, out=None, eps=CLIP_EPS, stream=None):
    """Multiplies the gradients by min(1, max_norm / (norm + eps)) and returns
    their norm before that (0-d fp32).

    In place, or with out into tensors of the same shapes, whose types may be
    others (then the gradients are left as they are).  Tensors that are written
    must not overlap.  The norm is not checked: a NaN or infinity goes into the
    gradients (clip_grad_norm_ can raise instead)."""
    grads = list(grads)
    outs = grads if out is None else list(out)
    if len(outs) != len(grads):
        raise ValueError(f"out must have one tensor for each of the {len(grads)} gradients, got {len(outs)}")
    code = _norm_code(norm_type)
    max_norm = float(max_norm)
    if not max_norm >= 0.0:
        raise ValueError(f"max_norm must be at least 0, got {max_norm}")
    if not grads:
        return torch.zeros(())
    return _call(grads, outs, code, max_norm, float(eps), stream)


def clip_grad_norm_(parameters, max_norm, norm_type=2.0, error_if_nonfinite=False):
    """Clips the gradients of the parameters (a tensor or several; those
    without a gradient are passed over) in place and returns their norm.

    error_if_nonfinite waits for the norm and raises RuntimeError, the
    gradients untouched, when it is NaN or infinite."""
    if isinstance(parameters, torch.Tensor):
        parameters = [parameters]
    grads = [p.grad for p in parameters if p.grad is not None]
    if error_if_nonfinite:
        norm = cce_grad_norm(grads, norm_type)
        if not math.isfinite(norm.item()):
            raise RuntimeError(f"the total norm of the gradients is {norm.item()}: they are not clipped")
    return cce_clip_grads(grads, max_norm, norm_type)
