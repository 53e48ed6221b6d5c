"""64-bit references of the layers in front of the head, and error bounds.

Bounds, fixed before any run.  Products of 16-bit values are exact in fp32.  A
tensor core adds 16 of them to its fp32 accumulator at a time and may cut where it
could round: an addition loses at most 2^-22 of the magnitudes it has seen, and
there are K / 16 of them, up to 4 inside of a step and up to 72 more where K is
split and joined or shared between warps, so a sum is off by at most
(K / 16 + 76) * 2^-22 of the sum of absolute products.  An activation passes that
on with a slope of at most 1.13, and adds errors of its own functions: e^-z with
2 ulp and the ulp of its rounded argument, |z| * 2^-24 on top (z / (1 + e^-z) is
below 2^-24 where |z| > 20 is negative), divisions with 2 ulp, erfc with 5:
2^-18 of |z| bounds them all.  Slopes (the derivative) are bounded in their own
right by 1.13, are off by the same 2^-18 absolute, and change by at most 1.13 per
unit of z.  A result is rounded once to its type: u = finfo.eps / 2 relative, or
half of the smallest subnormal."""
from __future__ import annotations

import math

import torch

ACTS = (None, "relu", "gelu", "gelu_tanh", "silu")
FUNC = 2.0 ** -18
C = math.sqrt(2 / math.pi)


def act64(name, z):
    if name is None:
        return z
    if name == "relu":
        return z.clamp(min=0)
    if name == "gelu":
        return z * 0.5 * torch.special.erfc(-z / math.sqrt(2))
    if name == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(C * (z + 0.044715 * z ** 3)))
    return z * torch.sigmoid(z)


def slope64(name, z):
    if name is None:
        return torch.ones_like(z)
    if name == "relu":
        return (z > 0).double()
    if name == "gelu":
        return 0.5 * torch.special.erfc(-z / math.sqrt(2)) + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    if name == "gelu_tanh":
        t = torch.tanh(C * (z + 0.044715 * z ** 3))
        return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * C * (1 + 3 * 0.044715 * z * z)
    s = torch.sigmoid(z)
    return s * (1 + z * (1 - s))


def steps(K):
    return (K / 16 + 76) * 2.0 ** -22


def half_step(ref, dtype):
    """Half a step at most; int16 stands for what the forward keeps: 9 bits of fraction, down to 2^-30."""
    eps, least = (2.0 ** -9, 2.0 ** -30) if dtype == torch.int16 else (torch.finfo(dtype).eps, torch.finfo(dtype).smallest_normal)
    return ref.abs() * (eps / 2) + least * eps / 2


def kept(words):
    """The values of what a forward keeps for its backward: sign, 6 bits of exponent (bias 31), 9 of fraction."""
    if words.dtype != torch.int16:
        return words.double()
    w = words.to(torch.int64) & 0xFFFF
    exponent, fraction = (w >> 9) & 63, (w & 511).double()
    power = torch.tensor([2.0 ** (e - 31) for e in range(64)], dtype=torch.float64, device=w.device)
    v = torch.where(exponent == 0, fraction * 2.0 ** -39, (1 + fraction / 512) * power[exponent])
    v = torch.where(exponent == 63, torch.where(fraction == 0, math.inf, math.nan), v)
    return torch.where(w >= 0x8000, -v, v)


def within_kept(words, ref, slack, what=""):
    tol = half_step(ref.abs() + slack, words.dtype) + slack
    assert ((kept(words) - ref).abs() <= tol).all(), what


def within(got, ref, slack, what=""):
    """|got - ref| <= the rounding to got's type + slack, element by element."""
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    tol = half_step(ref.abs() + slack, got.dtype) + slack
    bad = ~((got.double() - ref).abs() <= tol)
    if bad.any():
        at = tuple(bad.nonzero()[0].tolist())
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} outside, first at {at}: {got[at].item()} for "
                             f"{ref[at].item()} +- {tol[at].item()}")


def product(x, w):
    """(x w^T, the bound of its error) in 64 bits."""
    x, w = x.double(), w.double()
    return x @ w.T, (x.abs() @ w.abs().T) * steps(x.shape[-1])


def linear(x, w, b=None, r=None, act=None):
    """(y, its slack, z, its slack)."""
    z, dz = product(x, w)
    if b is not None:
        z = z + b.double()
        dz = dz + z.abs() * 2.0 ** -24 + b.double().abs() * 2.0 ** -24
    y = act64(act, z)
    dy = 1.13 * dz + (FUNC * z.abs() if act else 0.0)
    if r is not None:
        y = y + r.double()
        dy = dy + (y.abs() + r.double().abs()) * 2.0 ** -23
    return y, dy, z, dz


def gated(x, wg, wu, act):
    g, dg = product(x, wg)
    u, du = product(x, wu)
    a = act64(act, g)
    da = 1.13 * dg + (FUNC * g.abs() if act else 0.0)
    y = a * u
    return y, da * (u.abs() + du) + a.abs() * du + y.abs() * 2.0 ** -23, (g, dg), (u, du)


def grad_out(g, z, act):
    """(g act'(z), the slack) where z is what the kernel reads."""
    s = slope64(act, z.double())
    g = g.double()
    return g * s, g.abs() * (FUNC * (1.0 + z.double().abs()) if act else 0.0) + (g * s).abs() * 2.0 ** -23


def backward_products(dzs, slacks, x, ws, dtype):
    """dx and the dw from the gradients in front of the activation, which the
    kernel rounds to the operands' type: ((dx, slack), [(dw, slack)])."""
    x = x.double()
    dx = sum(d @ w.double() for d, w in zip(dzs, ws))
    off = [half_step(d.abs() + s, dtype) + s for d, s in zip(dzs, slacks)]
    n = dzs[0].shape[-1] * len(dzs)
    m = dzs[0].shape[0]
    dx_slack = sum(o @ w.double().abs() + (d.abs() + o) @ w.double().abs() * steps(n) for d, o, w in zip(dzs, off, ws))
    dws = [(d.T @ x, o.T @ x.abs() + (d.abs() + o).T @ x.abs() * steps(m)) for d, o in zip(dzs, off)]
    return (dx, dx_slack), dws
