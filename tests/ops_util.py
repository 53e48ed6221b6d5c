"""Helpers of the GPU tests of the norms: 64-bit references and error bounds.

Bounds, fixed before any run.  A result is its fp32 value rounded once to its
type: at most u_T = finfo(T).eps / 2 relative (plus half the smallest
subnormal).  The fp32 value itself differs from the 64-bit one by its
roundings of 2^-24: every sum here is added in chains of at most 180 terms one
after another (registers of a thread, shuffles, warps, blocks), and a value
passes through at most three of them, each multiplied by the sum of absolute
values.  512 * 2^-24 = 2^-15 of that magnitude bounds it."""
from __future__ import annotations

import numpy as np
import torch

U32 = 512 * 2.0 ** -24


def f64(t):
    return t.detach().double().cpu().numpy().reshape(-1, t.shape[-1])


def within(got, ref, magnitude, dtype, what=""):
    """|got - ref| <= rounding to dtype + U32 * magnitude, element by element."""
    got = got.detach().double().cpu().numpy().reshape(ref.shape)
    fi = torch.finfo(dtype)
    slack = U32 * magnitude
    tol = (fi.eps / 2) * (np.abs(ref) + slack) + slack + fi.smallest_normal * fi.eps / 2
    bad = ~(np.abs(got - ref) <= tol)
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.size} outside, first at {np.argwhere(bad)[0]}: "
                           f"{got[bad][0]} for {ref[bad][0]} +- {np.broadcast_to(tol, ref.shape)[bad][0]}")


def forward_magnitude(x, gain, bias, mean, rstd):
    """Of the terms of y: x - mean is off by roundings of |x| and mean|x|; the
    standard deviation by as much, which z multiplies."""
    m = np.abs(x) + (np.abs(x).mean(axis=1, keepdims=True) if np.any(mean) else 0.0)
    z = np.abs(x - mean[:, None]) * rstd[:, None]
    return (m + z * m.max(axis=1, keepdims=True)) * rstd[:, None] * np.abs(gain) + np.abs(bias)


def backward_magnitudes(dy, x, gain, mean, rstd, layer):
    z = (np.abs(x) + np.abs(mean)[:, None]) * rstd[:, None]
    g = np.abs(dy * gain)
    dx = g + z * (g * z).mean(axis=1, keepdims=True) + (g.mean(axis=1, keepdims=True) if layer else 0.0)
    return dx * rstd[:, None], (np.abs(dy) * z).sum(axis=0), np.abs(dy).sum(axis=0)
