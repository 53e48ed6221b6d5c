"""Layer norm and RMS norm: the norm that produces the classifier head's
hidden states, forward and backward, on the library's CUDA kernels.

    y = layer_norm(x, weight, bias)          # last dimension; differentiable
    y = rms_norm(x, weight, weight_offset=1.0)
    loss = linear_cross_entropy(y, C, targets)

x is bf16, fp16 or fp32 with any number of leading dimensions; the result has
x's type, or with out_dtype a 16-bit type from fp32 rows.  Arithmetic and the
saved statistics are fp32.  Rows may be strided (hidden[:, :-1] is read in
place); the result is contiguous.  Calls run on the current stream of x's
device and can be captured into a CUDA graph (a backward pass while no graph of
autograd that was made outside of the capture holds the same leaves: torch ties
their accumulation to the stream of the first).  Arguments that do not fit
raise ValueError, a status of the library CCEError.  Forward-mode derivatives and
tracing (torch.jit.trace, make_fx) raise NotImplementedError.
"""
from __future__ import annotations

import torch

from . import _lib, _native

_rows = _native.rows


def norm_backward_workspace_bytes(N, D) -> int:
    return int(_lib.load().cce_norm_backward_workspace_bytes(N, D))


def cce_layer_norm_forward(x, weight=None, bias=None, eps=1e-5, *, out_dtype=None, stats=True, stream=None):
    """(y, mean, rstd) of a layer norm over the last dimension; mean and rstd
    are fp32 with one value a row, None with stats=False."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return _native.layer_norm_forward(x, weight, bias, eps, out_dtype, stats)
    return _native.layer_norm_forward(x, weight, bias, eps, out_dtype, stats)


def cce_rms_norm_forward(x, weight=None, eps=1e-6, *, weight_offset=0.0, out_dtype=None, stats=True, stream=None):
    """(y, rstd) of an RMS norm over the last dimension: y = x * rstd *
    (weight_offset + weight); rstd is None with stats=False."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return _native.rms_norm_forward(x, weight, eps, weight_offset, out_dtype, stats)
    return _native.rms_norm_forward(x, weight, eps, weight_offset, out_dtype, stats)


def cce_layer_norm_backward(grad_y, x, weight, mean, rstd, *, need_dx=True, need_dweight=True, need_dbias=True,
                            param_dtype=None, stream=None):
    """(dx, dweight, dbias) of a layer norm whose forward gave mean and rstd;
    None for those not needed.  The parameters' gradients have the weight's
    type, or param_dtype where there is no weight (x's type if not given)."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return _native.layer_norm_backward(grad_y, x, weight, mean, rstd, need_dx, need_dweight, need_dbias,
                                               param_dtype)
    return _native.layer_norm_backward(grad_y, x, weight, mean, rstd, need_dx, need_dweight, need_dbias, param_dtype)


def cce_rms_norm_backward(grad_y, x, weight, rstd, *, weight_offset=0.0, need_dx=True, need_dweight=True,
                          stream=None):
    """(dx, dweight) of an RMS norm whose forward gave rstd; None for those
    not needed (dweight also where there is no weight)."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return _native.rms_norm_backward(grad_y, x, weight, rstd, weight_offset, need_dx, need_dweight)
    return _native.rms_norm_backward(grad_y, x, weight, rstd, weight_offset, need_dx, need_dweight)


def layer_norm(x, weight=None, bias=None, eps=1e-5, out_dtype=None):
    """Layer norm over x's last dimension: (x - mean) / sqrt(var + eps) *
    weight + bias, differentiable in x, weight and bias (once).

    weight and bias [D] are optional and share one type, which may differ from
    x's.  out_dtype: a 16-bit result from float32 rows (default: x's type)."""
    return _native.layer_norm(x, weight, bias, eps, out_dtype)


def rms_norm(x, weight=None, eps=1e-6, weight_offset=0.0, out_dtype=None):
    """RMS norm over x's last dimension: x / sqrt(mean(x^2) + eps) *
    (weight_offset + weight), differentiable in x and weight (once).

    weight_offset is 1 for models that store the weight minus one (without a
    weight there is no factor).  out_dtype as for layer_norm."""
    return _native.rms_norm(x, weight, eps, weight_offset, out_dtype)
