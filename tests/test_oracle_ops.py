"""Pins of the fp64 oracle of the norms and of clipping, each independent of
the oracle's own formulas: closed forms, torch's fp64 autograd, differences."""
import numpy as np
import pytest
import torch

from oracle import ops


def _case(seed, N=5, D=7):
    r = np.random.default_rng(seed)
    return r.normal(size=(N, D)) + 0.3, r.normal(size=D), r.normal(size=D), r.normal(size=(N, D))


@pytest.mark.parametrize("layer", [True, False])
def test_forward_and_gradients_equal_torch_autograd(layer):
    x, w, b, dy = _case(1)
    b = b if layer else np.zeros_like(b)
    eps = 1e-5
    mean, rstd = ops.norm_stats(x, eps, layer)
    y = ops.norm_forward(x, w, b, mean, rstd)
    dx, dw, db = ops.norm_backward(dy, x, w, mean, rstd, layer)
    xt, wt, bt = (torch.tensor(v, requires_grad=True) for v in (x, w, b))
    if layer:
        yt = torch.nn.functional.layer_norm(xt, (x.shape[1],), wt, bt, eps)
    else:
        yt = xt * torch.rsqrt(xt.square().mean(-1, keepdim=True) + eps) * wt
    grads = torch.autograd.grad(yt, (xt, wt) + ((bt,) if layer else ()), torch.tensor(dy))
    for ours, theirs in zip((y, dx, dw, db), (yt.detach(),) + grads):
        np.testing.assert_allclose(ours, theirs.numpy(), rtol=1e-11, atol=1e-12)


@pytest.mark.parametrize("layer", [True, False])
def test_gradient_equals_differences(layer):
    """Central differences of sum(dy * y) for every entry of x, gain and bias."""
    x, w, b, dy = _case(2, 3, 5)
    eps, h = 1e-5, 1e-6

    def f(x, w, b):
        return float((dy * ops.norm_forward(x, w, b, *ops.norm_stats(x, eps, layer))).sum())

    dx, dw, db = ops.norm_backward(dy, x, w, *ops.norm_stats(x, eps, layer), layer)
    for which, grad in enumerate((dx, dw, db)):
        for at in np.ndindex(grad.shape):
            lo, hi = [v.copy() for v in (x, w, b)], [v.copy() for v in (x, w, b)]
            lo[which][at] -= h
            hi[which][at] += h
            assert (f(*hi) - f(*lo)) / (2 * h) == pytest.approx(grad[at], rel=1e-6, abs=1e-7)


def test_closed_forms():
    mean, rstd = ops.norm_stats(np.array([[1.0, 3.0]]), 0.0, True)
    assert mean[0] == 2.0 and rstd[0] == 1.0
    _, rstd = ops.norm_stats(np.array([[3.0, 4.0]]), 0.0, False)
    assert rstd[0] == pytest.approx(np.sqrt(2) / 5)
    assert ops.global_norm([np.array([3.0]), np.array([[4.0]])]) == 5.0
    assert ops.global_norm([np.array([3.0]), np.array([[-4.0]])], np.inf) == 4.0
    assert ops.global_norm([]) == 0.0
    assert ops.clip_factor(1.0, 2.0) == 1.0
    assert ops.clip_factor(4.0, 2.0, eps=0.0) == 0.5


def test_a_planted_mistake_is_seen():
    """Dropping the mean's own gradient, as an RMS norm's backward does, fails the layer norm's pin."""
    x, w, _, dy = _case(3)
    mean, rstd = ops.norm_stats(x, 1e-5, True)
    right = ops.norm_backward(dy, x, w, mean, rstd, True)[0]
    wrong = ops.norm_backward(dy, x, w, mean, rstd, False)[0]
    assert np.abs(right - wrong).max() > 1e-2
