"""Gradients through a relu whose inputs are small or large: its slope is 1 for every positive one."""
import pytest
import torch

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def cce():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    from tests.conftest import build_library
    build_library()
    import linear_cross_entropy_gb300
    yield linear_cross_entropy_gb300
    linear_cross_entropy_gb300.raise_pending_errors()


@pytest.mark.parametrize("M,N,K", [(3, 40, 8), (64, 136, 72), (100, 33, 65)])
@pytest.mark.parametrize("size", [2.0 ** -100, 2.0 ** -42, 2.0 ** -39, 1.0, 2.0 ** 33, 2.0 ** 60])
@pytest.mark.parametrize("out", [None, F32])
def test_slope(cce, M, N, K, size, out):
    """One input of a row is 1, the others 0: every z is a weight, exact in any sum."""
    gen = torch.Generator(device="cuda").manual_seed(1)
    x = torch.zeros(M, K, device="cuda", dtype=BF16)
    x[torch.arange(M), torch.arange(M) % K] = 1.0
    w = (size * torch.randn(N, K, generator=gen, device="cuda")).to(BF16)
    g = torch.randn(M, N, generator=gen, device="cuda").to(out or BF16)
    xs, ws, b = x.clone().requires_grad_(), w.clone().requires_grad_(), torch.zeros(N, device="cuda", requires_grad=True)
    y = cce.linear(xs, ws, b, activation="relu", out_dtype=out)
    z = x.double() @ w.double().T
    assert torch.equal(y.double(), z.clamp(min=0).to(y.dtype).double())
    y.backward(g)
    dz = g.double() * (z > 0)
    # sums of M values in fp32, each off by 2^-24 of the magnitudes
    assert ((b.grad.double() - dz.sum(0)).abs() <= M * 2.0 ** -24 * dz.abs().sum(0)).all()
    # dz is rounded to bf16, its sum with ones and zeros is fp32 and rounded to bf16 once more
    dw, most = dz.T @ x.double(), dz.abs().T @ x.double()
    assert ((ws.grad.double() - dw).abs() <= 2.0 ** -8 * most + 2.0 ** -8 * dw.abs() + 2.0 ** -20 * most).all()
    assert ((ws.grad != 0) == (dw != 0)).all() or M > K  # sums of several may cancel
