"""Clipping where the factor's quotient is no number: an infinite norm below an
infinite limit, and a norm and a limit of 0 without eps."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def cce():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    from tests.conftest import build_library
    build_library()
    import linear_cross_entropy_gb300
    return linear_cross_entropy_gb300


def _gradients(dtype, value):
    dense = torch.arange(5000, device="cuda").to(dtype)
    dense[77] = value
    cut = torch.ones(30, 40, device="cuda", dtype=dtype)[:, 3:17]  # not one block of memory
    return [dense, cut]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("norm_type", [2.0, math.inf])
@pytest.mark.parametrize("value", [math.inf, -math.inf])
def test_no_limit_leaves_infinities_alone(cce, dtype, norm_type, value):
    grads = _gradients(dtype, value)
    before = [g.clone() for g in grads]
    outs = [torch.empty(g.shape, device="cuda") for g in grads]
    assert cce.cce_clip_grads(grads, math.inf, norm_type, out=outs).item() == math.inf
    assert all(torch.equal(o, b.float()) for o, b in zip(outs, before))
    assert cce.cce_clip_grads(grads, math.inf, norm_type).item() == math.inf
    assert all(torch.equal(g, b) for g, b in zip(grads, before))


def test_a_norm_beyond_fp32_without_a_limit(cce):
    big = [torch.full((64,), 3e38, device="cuda")]
    assert cce.cce_clip_grads(big, math.inf).item() == math.inf
    assert torch.equal(big[0], torch.full_like(big[0], 3e38))


@pytest.mark.parametrize("limit", [0.0, 1.0, math.inf])
def test_zeros_without_eps(cce, limit):
    zeros = [torch.zeros(5000, device="cuda"), torch.zeros(30, 40, device="cuda")[:, 3:17]]
    outs = [torch.full(z.shape, 7.0, device="cuda") for z in zeros]
    assert cce.cce_clip_grads(zeros, limit, out=outs, eps=0.0).item() == 0.0
    cce.cce_clip_grads(zeros, limit, eps=0.0)
    assert not any(t.any() for t in zeros + outs)


@pytest.mark.parametrize("limit", [0.0, 1.0, math.inf])
def test_a_nan_goes_everywhere(cce, limit):
    grads = _gradients(torch.float32, math.nan)
    assert math.isnan(cce.cce_clip_grads(grads, limit).item())
    assert all(torch.isnan(g).all() for g in grads)


@pytest.mark.parametrize("limit", [0.0, 1.0])
def test_a_limit_below_an_infinite_norm_is_factor_0(cce, limit):
    grads = _gradients(torch.float32, math.inf)
    cce.cce_clip_grads(grads, limit)
    assert torch.isnan(grads[0][77]) and not torch.nan_to_num(grads[0]).any() and not grads[1].any()
