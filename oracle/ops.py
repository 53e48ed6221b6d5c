"""fp64 CPU oracle of the operators around the head: layer norm, RMS norm,
the global gradient norm and clipping, from their formulas.

TEST INFRASTRUCTURE ONLY, like the rest of this package; it imports nothing
from the product.  Arrays are float64 [N, D] (rows first).
"""
from __future__ import annotations

import numpy as np


def norm_stats(x, eps, layer):
    """(mean, rstd), each [N]; mean is 0 for RMS norm."""
    mean = x.mean(axis=1) if layer else np.zeros(x.shape[0])
    var = ((x - mean[:, None]) ** 2).mean(axis=1)
    return mean, 1.0 / np.sqrt(var + eps)


def norm_forward(x, gain, bias, mean, rstd):
    """z * gain + bias with z = (x - mean) * rstd."""
    return (x - mean[:, None]) * rstd[:, None] * gain + bias


def norm_backward(dy, x, gain, mean, rstd, layer):
    """(dx, dgain, dbias) by the chain rule through z, mean and rstd."""
    z = (x - mean[:, None]) * rstd[:, None]
    g = dy * gain
    dx = g - z * (g * z).mean(axis=1, keepdims=True)
    if layer:
        dx = dx - g.mean(axis=1, keepdims=True)
    return dx * rstd[:, None], (dy * z).sum(axis=0), dy.sum(axis=0)


def global_norm(tensors, norm_type=2.0):
    """The norm of all values of all tensors together."""
    flat = np.concatenate([np.asarray(t, dtype=np.float64).ravel() for t in tensors] or [np.zeros(0)])
    if np.isinf(norm_type):
        return float(np.abs(flat).max()) if flat.size else 0.0
    return float(np.sqrt((flat ** 2).sum()))


def clip_factor(norm, max_norm, eps=1e-6):
    """min(1, max_norm / (norm + eps)); NaN for a NaN norm, 1 where the quotient is infinity by infinity or 0 by 0."""
    if np.isnan(norm):
        return float("nan")
    with np.errstate(invalid="ignore", divide="ignore"):
        return float(np.fmin(1.0, np.float64(max_norm) / np.float64(norm + eps)))
