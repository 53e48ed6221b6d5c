"""The global norm of many gradients and clipping by it, on the library's CUDA
kernels: a launch covers up to 1000 tensors of any sizes and types, and nothing
waits for the GPU.

    loss.backward()
    norm = clip_grad_norm_(model.parameters(), 1.0)  # 0-d fp32, before clipping

cce_clip_grads writes the clipped gradients in place or into other tensors
(say, the 32-bit buffers of an optimiser).  Calls run on the current stream of
the gradients' device and can be captured into a CUDA graph.  Tensors with a
forward-mode tangent and tracing (torch.jit.trace, make_fx) raise
NotImplementedError.
"""
from __future__ import annotations

import math

import torch

from . import _lib, _native

CLIP_EPS = 1e-6  # added to the norm before the division

_dims = _native.dims


def grad_norm_workspace_bytes(n_dense, n_strided=0) -> int:
    return int(_lib.load().cce_grad_norm_workspace_bytes(n_dense, n_strided))


def _norm_code(norm_type):
    norm_type = float(norm_type)
    if norm_type == 2.0:
        return 2
    if norm_type == math.inf:
        return 0
    raise ValueError(f"norm_type must be 2 or infinity, got {norm_type}")


def cce_grad_norm(grads, norm_type=2.0, *, stream=None):
    """The norm (0-d fp32) over all values of the tensors together: 2 or
    infinity.  Without tensors it is a 0 on the CPU."""
    grads = list(grads)
    code = _norm_code(norm_type)
    if not grads:
        return torch.zeros(())
    if stream is not None:
        with torch.cuda.stream(stream):
            return _native.grad_norm(grads, code)
    return _native.grad_norm(grads, code)


def cce_clip_grads(grads, max_norm, norm_type=2.0, *, out=None, eps=CLIP_EPS, stream=None):
    """Multiplies the gradients by min(1, max_norm / (norm + eps)) and returns
    their norm before that (0-d fp32).

    In place, or with out into tensors of the same shapes, whose types may be
    others (then the gradients are left as they are).  Tensors that are written
    must not overlap.  The norm is not checked: a NaN goes into the gradients, an
    infinity makes them 0 and itself NaN, unless max_norm is infinite too
    (clip_grad_norm_ can raise instead)."""
    grads = list(grads)
    if out is not None:
        out = list(out)
        if len(out) != len(grads):
            raise ValueError(f"out must have one tensor for each of the {len(grads)} gradients, got {len(out)}")
    code = _norm_code(norm_type)
    max_norm = float(max_norm)
    if not max_norm >= 0.0:
        raise ValueError(f"max_norm must be at least 0, got {max_norm}")
    if not grads:
        return torch.zeros(())
    if stream is not None:
        with torch.cuda.stream(stream):
            return _native.clip_grads(grads, out, code, max_norm, eps)
    return _native.clip_grads(grads, out, code, max_norm, eps)


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
