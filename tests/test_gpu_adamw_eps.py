"""AdamW with an eps among fp32's subnormal values: it is not 0.

Bounds, fixed before any run, as in test_gpu_adamw, and half of the least subnormal for an m
among them."""
import pytest
import torch

from tests import test_gpu_adamw as A

pytestmark = pytest.mark.gpu

F32 = torch.float32
EPS = [1e-38, 1e-40, 3e-44]  # one normal value's neighbour and two subnormals


@pytest.fixture(scope="module", autouse=True)
def cce():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    from tests.conftest import build_library
    build_library()
    import linear_cross_entropy_gb300
    return linear_cross_entropy_gb300


@pytest.mark.parametrize("eps", EPS)
@pytest.mark.parametrize("offset", [0, 1])
@pytest.mark.parametrize("dtype", [A.BF16, F32])
def test_values_without_a_gradient_stay(cce, eps, offset, dtype):
    """m = v = g = 0: the update is 0 / eps, nothing but the decay."""
    for master in (False, True):
        p, _, _, _ = A.make(1, [(300,), (5, 7)], dtype, dtype, offset)
        masters = [t.float().clone() for t in p] if master else None
        zeros = [torch.zeros_like(t) for t in p]
        want = [(t.float() * (1 - 1e-2 * 0.1)).to(dtype) for t in p]
        m, v = ([torch.zeros_like(t, dtype=F32) for t in p] for _ in "mv")
        q = [t.clone() for t in p]
        cce.cce_adamw_step(p, zeros, m, v, 1, lr=1e-2, eps=eps, weight_decay=0.1, masters=masters)
        for a, b in zip(p, want):
            assert ((a - b).abs() <= torch.finfo(dtype).eps * b.abs()).all()
        masters = [t.float().clone() for t in q] if master else None
        cce.cce_adamw8_step(q, zeros, *A.eight_bit_state(cce, q), 1, lr=1e-2, eps=eps, weight_decay=0.1, masters=masters)
        for a, b in zip(q, p):
            assert torch.equal(a, b)


@pytest.mark.parametrize("eps", EPS)
@pytest.mark.parametrize("on_device", [False, True])
def test_its_size_counts(cce, eps, on_device):
    """v = g = 0 and an m of the size of eps: the step is lr m / eps; with a root far above it, eps does not matter."""
    n = 64
    p, g, m = (torch.full((n,), value, device="cuda") for value in (0.0, 0.0, 2 * eps))
    m[1::2] *= -1
    v = torch.zeros(n, device="cuda")
    m[n // 2:], v[n // 2:] = 1e-3, 1e-4
    w1, _, _, w_terms, _ = A.reference(p.double(), g, m.double(), v.double(), 3, 1e-3, (0.9, 0.99), eps, 0.0)
    # m1, 1.8 eps, is rounded to a multiple of 2^-149
    off = 2.0 ** -150 / eps
    step = torch.tensor(3, device="cuda") if on_device else 3
    cce.cce_adamw_step([p], [g], [m], [v], step, lr=1e-3, betas=(0.9, 0.99), eps=eps, weight_decay=0.0)
    tol = (2.0 ** -19 + off) * w_terms
    assert ((p.double() - w1).abs() <= tol).all(), (p[:4], w1[:4], tol[:4])
