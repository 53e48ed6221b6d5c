"""fp32 results of few rows over a long K: sums go on in parts.

Bound, fixed before any run, as for many rows: eight warps share K, and a warp's sum goes on in other registers every 1,024
of its k, so that beyond 8,192 a sum's error is its parts', relative to the norm that of K = 8,192 (parts' errors grow
together as their sums do), where one accumulator's would grow with K.  Twice is allowed, and 2^-24 for each of the
additions of parts."""
import pytest
import torch

pytestmark = pytest.mark.gpu

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def cce():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    from tests.conftest import build_library
    build_library()
    import linear_cross_entropy_gb300
    yield linear_cross_entropy_gb300
    linear_cross_entropy_gb300.raise_pending_errors()


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("M", [1, 9, 32])
def test_few_rows(cce, M, dtype):
    gen = torch.Generator(device="cuda").manual_seed(1)
    off = []
    for K in (8192, 8192 + 512, 65536 + 72, 300000 + 5):
        x, w = (torch.randn(rows, K, generator=gen, device="cuda").to(dtype) for rows in (M, 300))
        ref = x.double() @ w.double().T
        off.append(((cce.linear(x, w, out_dtype=F32) - ref).norm() / ref.norm()).item())
        assert off[-1] < 2 * off[0] + (K / 8192 + 2) * 2.0 ** -24, (K, off)


@pytest.mark.parametrize("M", [1, 9, 32])
def test_parts_count_once(cce, M):
    """Ones: every sum is K, exact in fp32 in any order; a gated layer's two sums as well."""
    for K in (8192, 8192 + 64, 16384, 16384 + 8, 16384 + 1024 + 8, 65536 + 8):
        x = torch.ones(M, K, device="cuda", dtype=BF16)
        w = torch.ones(40, K, device="cuda", dtype=BF16)
        assert (cce.linear(x, w, out_dtype=F32) == K).all()
        assert (cce.gated_linear(x * 2.0 ** -8, w * 2.0 ** -8, w, None) == torch.tensor(float(K) * K * 2.0 ** -24).bfloat16().item()).all()
