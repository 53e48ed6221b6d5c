"""The bounds of the norms (tests/norm_bounds.py) on the CPU: an emulation of the
kernels' arithmetic in fp32 is inside them, and mistakes planted in it are not,
with rows whose mean is 1, 10 and 1000 deviations from 0."""
import numpy as np
import pytest
import torch

from tests import norm_bounds as B

F = np.float32
EPS = 1e-5


def _inputs(seed, N, D, mean):
    r = np.random.default_rng(seed)
    return ((r.normal(size=(N, D)) + mean).astype(F), (1 + 0.3 * r.normal(size=D)).astype(F),
            (0.3 * r.normal(size=D)).astype(F), r.normal(size=(N, D)).astype(F))


def _stats(x, one_pass=False):
    mean = x.mean(axis=1, dtype=F)
    var = (x * x).mean(axis=1, dtype=F) - mean * mean if one_pass else ((x - mean[:, None]) ** 2).mean(axis=1, dtype=F)
    return mean, (F(1) / np.sqrt(np.maximum(var, F(0)) + F(EPS))).astype(F)


def _z(x, mean, rstd, fused=False):
    if not fused:
        return (x - mean[:, None]) * rstd[:, None]
    shift = -mean * rstd  # rounded, then x rstd + shift rounded once
    return (x.astype(np.float64) * rstd[:, None] + shift[:, None]).astype(F)


def _grads(dy, x, w, mean, rstd, fused=False, no_centre=False, no_along=False):
    z = _z(x, mean, rstd, fused)
    g = dy * w
    dx = g.copy()
    if not no_centre:
        dx -= g.mean(axis=1, dtype=F, keepdims=True)
    if not no_along:
        dx -= z * (g * z).mean(axis=1, dtype=F, keepdims=True)
    return dx * rstd[:, None], (dy * z).sum(axis=0, dtype=F)


def _d(*arrays):
    return [a.astype(np.float64) for a in arrays]


@pytest.mark.parametrize("mean", [0.0, 1.0, 10.0, 1000.0])
@pytest.mark.parametrize("N,D", [(1, 100), (6, 896), (40, 1001), (6, 30000)])
def test_the_kernels_arithmetic_is_inside(N, D, mean):
    x, w, b, dy = _inputs(N + D, N, D, mean)
    m, r = _stats(x)
    y = _z(x, m, r) * w + b
    dx, dw = _grads(dy, x, w, m, r)
    x, w, b, dy, m, r, y, dx, dw = _d(x, w, b, dy, m, r, y, dx, dw)
    assert B.stats_outside(m, r, x, EPS, True) == (0, 0)
    assert B.y_outside(y, x, w, b, m, r, torch.float32) == 0
    assert B.grads_outside(dx, dw, dy, x, w, m, r, True, torch.float32, torch.float32) == (0, 0)


@pytest.mark.parametrize("N,D", [(6, 896), (40, 1001), (6, 30000)])
def test_a_variance_that_cancels_is_outside(N, D):
    x, *_ = _inputs(N + D, N, D, 1000.0)
    m, r = _d(*_stats(x, one_pass=True))
    assert B.stats_outside(m, r, x.astype(np.float64), EPS, True)[1] > 0


@pytest.mark.parametrize("mean", [0.0, 10.0, 1000.0])
@pytest.mark.parametrize("N,D", [(6, 896), (40, 1001), (6, 30000)])
@pytest.mark.parametrize("lost", ["no_centre", "no_along"])
def test_a_lost_term_of_dx_is_outside(N, D, mean, lost):
    x, w, b, dy = _inputs(N + D, N, D, mean)
    m, r = _stats(x)
    dx, dw = _grads(dy, x, w, m, r, **{lost: True})
    x, w, dy, m, r, dx, dw = _d(x, w, dy, m, r, dx, dw)
    assert B.grads_outside(dx, dw, dy, x, w, m, r, True, torch.float32, torch.float32)[0] > N * D // 2


@pytest.mark.parametrize("N,D,mean", [(1, 896, 10.0), (1, 896, 1000.0), (6, 1001, 10.0), (6, 1001, 1000.0),
                                      (40, 1001, 1000.0)])
def test_a_rounded_product_of_mean_and_rstd_is_outside(N, D, mean):
    x, w, b, dy = _inputs(N + D, N, D, mean)
    m, r = _stats(x)
    dx, dw = _grads(dy, x, w, m, r, fused=True)
    x, w, dy, m, r, dx, dw = _d(x, w, dy, m, r, dx, dw)
    bad = B.grads_outside(dx, dw, dy, x, w, m, r, True, torch.float32, torch.float32)[1]
    assert bad > (D // 2 if mean > 100 and N < 40 else 0)
