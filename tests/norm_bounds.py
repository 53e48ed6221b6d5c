"""Bounds of the norms that hold whatever the rows' mean, fixed before any run.

Each result is held against the 64-bit formula of what the call was given or
has itself returned: the statistics against x, y against x and the returned
statistics, the gradients against x and the given statistics.  So nothing is
multiplied by the size of the mean but the mean's own sum.

u = 2^-24.  A sum of n terms, each added to at most `depth` = min(n - 1, 180)
others in a chain (adding zeros is exact), is off by depth u of the sum of
their magnitudes.
  mean   the sum and a division: (depth + 2) u of mean |x|
  rstd   x - mean, its square, a sum, a division, eps: (depth + 5) u of the
         variance, of which the square root takes half, and 3 u for the root,
         the quotient and what is left: (depth / 2 + 6) u relative
  z      x - mean and the product with rstd: 2 u of |x - mean| rstd
  y      z, the gain (an offset rounds it once), product and sum: 6 u of |z gain| + |bias|
  dw     z, the product, the sum over N rows: (depth_N + 4) u of the sum of |dy z|
  dx     dy gain, z, both sums, 1 / D, products and sums: (depth_D + 12) u of
         rstd (|g| + mean |g| + |z| mean |g z|)
and every result is rounded once to its type."""
from __future__ import annotations

import numpy as np
import torch

u = 2.0 ** -24
TINY = 2.0 ** -140


def depth(n):
    return min(n - 1, 180)


def outside(got, ref, slack, dtype):
    """How many are further off than the slack and a rounding to dtype."""
    fi = torch.finfo(dtype)
    tol = (fi.eps / 2) * (np.abs(ref) + slack) + slack + fi.smallest_normal * fi.eps / 2 + TINY
    return int((~(np.abs(got - ref) <= tol)).sum())


def stats_outside(mean, rstd, x, eps, layer):
    """(means, rstds) outside; x [N, D] and the given statistics in 64 bits."""
    D = x.shape[1]
    d = depth(D)
    bad = outside(mean, x.mean(axis=1), (d + 2) * u * np.abs(x).mean(axis=1), torch.float32) if layer else 0
    want = 1.0 / np.sqrt(((x - mean[:, None]) ** 2).mean(axis=1) + eps)
    return bad, outside(rstd, want, (d / 2 + 6) * u * want, torch.float32)


def y_outside(y, x, gain, bias, mean, rstd, dtype):
    z = (x - mean[:, None]) * rstd[:, None]
    return outside(y, z * gain + bias, 6 * u * (np.abs(z * gain) + np.abs(bias)), dtype)


def grads_outside(dx, dw, dy, x, gain, mean, rstd, layer, x_type, p_type):
    """(dx, dw) outside."""
    N, D = x.shape
    z = (x - mean[:, None]) * rstd[:, None]
    g = dy * gain
    centre = g.mean(axis=1, keepdims=True) if layer else 0.0
    ref = rstd[:, None] * (g - centre - z * (g * z).mean(axis=1, keepdims=True))
    size = np.abs(g) + np.abs(z) * np.abs(g * z).mean(axis=1, keepdims=True)
    if layer:
        size = size + np.abs(g).mean(axis=1, keepdims=True)
    bad_x = outside(dx, ref, (depth(D) + 12) * u * rstd[:, None] * size, x_type)
    bad_w = outside(dw, (dy * z).sum(axis=0), (depth(N) + 4) * u * np.abs(dy * z).sum(axis=0), p_type)
    return bad_x, bad_w
