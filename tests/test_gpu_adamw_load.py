"""A checkpoint goes on in parameters of other strides."""
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


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_other_strides(cce, dtype):
    torch.manual_seed(1)
    a = torch.nn.Parameter(torch.randn(40, 33, device="cuda").to(dtype))
    g = torch.randn(40, 33, device="cuda").to(dtype)
    one = cce.AdamW([a], lr=1e-2, master_weights=True)
    a.grad = g
    one.step()
    b = torch.nn.Parameter(a.detach().t().contiguous().t())
    b.grad = g
    two = cce.AdamW([b], lr=1e-2, master_weights=True)
    two.load_state_dict(one.state_dict())
    for _ in range(2):
        one.step()
        two.step()
    assert torch.equal(a, b) and b.stride() == (1, 40)
    for k in ("exp_avg", "exp_avg_sq") + (("master",) if dtype != torch.float32 else ()):
        assert torch.equal(one.state[a][k], two.state[b][k])
