"""Layers in front of the classifier head on the library's tensor-core kernels:
a linear layer with bias, activation and residual in its epilogue, and the gated
product of a feed-forward block, forward and backward.

    h = linear(x, weight, bias, activation="gelu")            # a dense transform
    h = linear(x, weight, bias, residual=x, activation="silu")  # a prediction head
    a = gated_linear(rms_norm(x, g), gate_weight, up_weight)   # a feed-forward block
    x = linear(a, down_weight, residual=x)
    loss = linear_cross_entropy(rms_norm(x, g2), C, targets)

x and weights are bf16 or fp16 (one type), x with any number of leading
dimensions; products of them are summed in fp32, and everything behind the
product is fp32 with one rounding to the result.  The result is contiguous, of
x's type or float32.  x, weights and gradients may be strided: rows at one pitch,
on 16 bytes and a multiple of 8 elements apart, are read in place, others
(hidden[:, :-1], odd widths) are copied first.  Activations: None, "relu", "gelu"
(z Phi(z), Phi within (z^2 + 16) 2^-23 of itself), "gelu_tanh", "silu".  For the backward pass what goes into the
activation is kept in 16 bits, two of which more are fraction than bf16 has (torch
int16 words that only the backward reads; fp16 for fp16), and the gradient in front
of it is rounded to x's type for its products.  The words hold values from 2^-30 to
2^32 so, with fewer bits down to 2^-40; beyond, they count as infinite or 0 in the
backward pass: a bf16 gated layer whose gate or up projection passes 2^32 has a finite
result and an infinite or NaN gradient.  (linear with relu keeps x's type, whose sign
holds over all of its range.)

Calls run on the current stream of x's device and can be captured into a CUDA
graph (a backward pass while no graph of autograd that was made outside of the
capture holds the same leaves: torch ties their accumulation to the stream of the
first).  Arguments that do not fit raise ValueError, a status of the library
CCEError.  Forward-mode derivatives and tracing (torch.jit.trace, make_fx) raise
NotImplementedError, a derivative of a gradient RuntimeError.
"""
from __future__ import annotations

import torch

from . import _lib, _native


def _name(activation):
    return "none" if activation is None else activation


def linear_forward_workspace_bytes(M, N, K) -> int:
    return int(_lib.load().cce_linear_forward_workspace_bytes(M, N, K))


def linear_backward_workspace_bytes(M, N, K) -> int:
    return int(_lib.load().cce_linear_backward_workspace_bytes(M, N, K))


def gated_linear_forward_workspace_bytes(M, N, K) -> int:
    return int(_lib.load().cce_gated_linear_forward_workspace_bytes(M, N, K))


def gated_linear_backward_workspace_bytes(M, N, K) -> int:
    return int(_lib.load().cce_gated_linear_backward_workspace_bytes(M, N, K))


def _on(stream, call, *args):
    if stream is None:
        return call(*args)
    with torch.cuda.stream(stream):
        return call(*args)


def cce_linear_forward(x, weight, bias=None, residual=None, activation=None, *, out_dtype=None, save=False,
                       stream=None):
    """(y, z): y = act(z) + residual with z = x weight^T + bias.  z is for
    cce_linear_backward alone: int16 words for bf16, of the range above (a positive z
    below 2^-40 counts as 0, also for relu), else values of x's type; None with
    save=False or without activation."""
    return _on(stream, _native.linear_forward, x, weight, bias, residual, _name(activation), out_dtype, save)


def cce_linear_backward(grad_y, x, weight, z=None, activation=None, *, need_dx=True, need_dweight=True,
                        need_dbias=True, bias_dtype=None, stream=None):
    """(dx, dweight, dbias) of a linear layer whose forward gave z (or z in x's
    type); None for those not needed.  dbias has bias_dtype (x's type if not given).  The
    residual's gradient is grad_y."""
    return _on(stream, _native.linear_backward, grad_y, x, weight, z, _name(activation), need_dx, need_dweight,
               need_dbias, bias_dtype)


def cce_gated_linear_forward(x, gate_weight, up_weight, activation="silu", *, save=False, stream=None):
    """(y, gate, up): y = act(gate) * up with gate = x gate_weight^T and
    up = x up_weight^T.  gate and up are as z in cce_linear_forward, None with save=False."""
    return _on(stream, _native.gated_linear_forward, x, gate_weight, up_weight, _name(activation), save)


def cce_gated_linear_backward(grad_y, x, gate_weight, up_weight, gate, up, activation="silu", *, need_dx=True,
                              need_dgate_weight=True, need_dup_weight=True, stream=None):
    """(dx, dgate_weight, dup_weight) of a gated linear layer whose forward
    gave gate and up (or those in x's type); None for those not needed."""
    return _on(stream, _native.gated_linear_backward, grad_y, x, gate_weight, up_weight, gate, up, _name(activation),
               need_dx, need_dgate_weight, need_dup_weight)


def linear(x, weight, bias=None, residual=None, activation=None, out_dtype=None):
    """act(x weight^T + bias) + residual over x's last dimension, differentiable
    in the four tensors (once).

    x [..., K] and weight [N, K] bf16 or fp16; bias [N] of any of the three types;
    residual [..., N] of the result's type.  out_dtype: x's type (default) or
    float32."""
    return _native.linear(x, weight, bias, residual, _name(activation), out_dtype)


def gated_linear(x, gate_weight, up_weight, activation="silu"):
    """act(x gate_weight^T) * (x up_weight^T) over x's last dimension in one
    pass, differentiable in the three tensors (once).  Weights [N, K]; halves of
    one [2N, K] tensor are as good as two tensors."""
    return _native.gated_linear(x, gate_weight, up_weight, _name(activation))
