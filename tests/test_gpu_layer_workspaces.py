"""The layers' backward calls stay inside of the workspace that they ask for."""
import itertools

import pytest
import torch

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
CCE_F32, CCE_BF16, NONE, GELU, SILU = 0, 2, 0, 2, 4
DX, DW, DW_UP, DB, DZ = 1, 2, 4, 8, 16
GUARD = 4096


@pytest.fixture(scope="module", autouse=True)
def cce():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    from tests.conftest import build_library
    build_library()
    import linear_cross_entropy_gb300
    yield linear_cross_entropy_gb300
    linear_cross_entropy_gb300.raise_pending_errors()


@pytest.fixture(scope="module")
def lib(cce):
    from linear_cross_entropy_gb300 import _lib
    return _lib.load()


def guarded(need):
    """A workspace of `need` bytes (none where 16 are), and what lies behind it."""
    if need <= 16:
        return 0, torch.zeros(0, dtype=torch.uint8, device="cuda")
    whole = torch.full((need + GUARD,), 0xA5, dtype=torch.uint8, device="cuda")
    return whole.data_ptr(), whole[need:]


def pointer(t):
    return 0 if t is None else t.data_ptr()


SIZES = [(1, 8, 8), (40, 264, 72), (300, 640, 200), (4096, 136, 72), (100, 4096, 2048), (64, 20000, 64)]


@pytest.mark.parametrize("M,N,K", SIZES)
@pytest.mark.parametrize("act,y_type", [(NONE, CCE_BF16), (NONE, CCE_F32), (GELU, CCE_BF16)])
def test_linear(cce, lib, M, N, K, act, y_type):
    torch.manual_seed(1)
    x, w, z = (torch.randn(s, device="cuda").to(BF16) for s in ((M, K), (N, K), (M, N)))
    g = torch.randn(M, N, device="cuda").to(F32 if y_type == CCE_F32 else BF16)
    want = cce.cce_linear_backward(g, x, w, z if act else None, "gelu" if act else None, bias_dtype=F32)
    for dx, dw, db in itertools.product((0, 1), repeat=3):
        out = [torch.empty_like(t) if on else None for t, on in zip(want, (dx, dw, db))]
        staged = DZ if (act or y_type == CCE_F32) and (dx or dw) else 0
        need = lib.cce_linear_backward_workspace_bytes_ex(M, N, K, DX * dx | DW * dw | DB * db | staged)
        ws, guard = guarded(need)
        assert lib.cce_linear_backward(g.data_ptr(), N, y_type, x.data_ptr(), K, w.data_ptr(), K, CCE_BF16, z.data_ptr(), N,
                                       CCE_BF16, act, M, N, K, *(pointer(t) for t in out), CCE_F32, ws, need,
                                       torch.cuda.current_stream().cuda_stream) == 0
        assert (guard == 0xA5).all()
        # sums of K may be split otherwise than in the call for all
        for a, b in zip(out, want):
            assert a is None or torch.allclose(a.float(), b.float(), rtol=2.0 ** -7, atol=2.0 ** -7 * b.float().abs().max().item())


@pytest.mark.parametrize("M,N,K", SIZES)
def test_gated(cce, lib, M, N, K):
    torch.manual_seed(2)
    x, w, u, g, z0, z1 = (torch.randn(s, device="cuda").to(BF16) for s in ((M, K), (N, K), (N, K), (M, N), (M, N), (M, N)))
    want = cce.cce_gated_linear_backward(g, x, w, u, z0, z1)
    for dx, dw, du in itertools.product((0, 1), repeat=3):
        out = [torch.empty_like(t) if on else None for t, on in zip(want, (dx, dw, du))]
        need = lib.cce_gated_linear_backward_workspace_bytes_ex(M, N, K, DX * dx | DW * dw | DW_UP * du)
        ws, guard = guarded(need)
        assert lib.cce_gated_linear_backward(g.data_ptr(), N, x.data_ptr(), K, w.data_ptr(), K, u.data_ptr(), K, CCE_BF16,
                                             z0.data_ptr(), N, z1.data_ptr(), N, CCE_BF16, SILU, M, N, K,
                                             *(pointer(t) for t in out), ws, need, torch.cuda.current_stream().cuda_stream) == 0
        assert (guard == 0xA5).all()
        for a, b in zip(out, want):
            assert a is None or torch.allclose(a.float(), b.float(), rtol=2.0 ** -7, atol=2.0 ** -7 * b.float().abs().max().item())


def test_memory_of_a_plain_backward(cce):
    """No more than the gradients and partial sums of a small product: dz is grad_y."""
    M, N, K = 32768, 4096, 256
    x, w, g = (torch.randn(s, device="cuda").to(BF16) for s in ((M, K), (N, K), (M, N)))
    torch.cuda.synchronize()
    torch.cuda.reset_peak_memory_stats()
    before = torch.cuda.memory_allocated()
    out = cce.cce_linear_backward(g, x, w, need_dbias=False)
    torch.cuda.synchronize()
    own = sum(t.numel() * 2 for t in out if t is not None)
    assert torch.cuda.max_memory_allocated() - before <= own + M * N  # dz is twice that
