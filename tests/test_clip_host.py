"""Host side of the gradient norm and clipping without a GPU: workspace,
refusals of the C ABI before any launch and of the Python binding."""
import ctypes
import math

import pytest
import torch


@pytest.fixture(scope="module")
def lib():
    from tests.conftest import build_library
    build_library()
    from linear_cross_entropy_gb300 import _lib
    return _lib.load()


FAKE = 1 << 20  # an aligned non-null host integer: never dereferenced, checks fail first
F32, F16, BF16 = 0, 1, 2


def _row(p=FAKE, q=None, n=100, it=BF16, ot=BF16):
    return (p, p if q is None else q, n, it + (ot << 8))


def _table(rows):
    flat = [v for r in rows for v in r]
    return (ctypes.c_int64 * max(1, len(flat)))(*flat)


def _strided(p=FAKE, q=FAKE, it=BF16, ot=BF16, size=(1, 1, 3, 5), si=(0, 0, 8, 1), so=(0, 0, 8, 1)):
    from linear_cross_entropy_gb300._lib import Strided
    four = ctypes.c_int64 * 4
    return (Strided * 1)(Strided(p, q, it, ot, four(*size), four(*si), four(*so)))


def _clip(lib, rows=None, strided=None, norm_type=2, max_norm=1.0, eps=1e-6, norm=FAKE, ws=FAKE, wsb=1 << 30, count=None,
          clip=True):
    rows = [_row()] if rows is None else rows
    t = _table(rows)
    n = len(rows) if count is None else count
    s = ctypes.addressof(strided) if strided is not None else 0
    ns = 1 if strided is not None else 0
    args = (ctypes.addressof(t), n, s, ns, norm_type)
    if clip:
        return lib.cce_clip_grads(*args, max_norm, eps, norm, ws, wsb, 0)
    return lib.cce_grad_norm(*args, norm, ws, wsb, 0)


def test_workspace(lib):
    assert lib.cce_grad_norm_workspace_bytes(0, 0) > 0
    one, many = lib.cce_grad_norm_workspace_bytes(1, 0), lib.cce_grad_norm_workspace_bytes(1000, 0)
    assert one == many and lib.cce_grad_norm_workspace_bytes(1001, 0) == 2 * one
    assert lib.cce_grad_norm_workspace_bytes(1, 3) == 4 * one
    assert lib.cce_grad_norm_workspace_bytes(-1, 0) == 0 and lib.cce_grad_norm_workspace_bytes(0, -1) == 0


@pytest.mark.parametrize("kw,status", [
    (dict(norm_type=1), 4), (dict(norm_type=-2), 4), (dict(norm=0), 1), (dict(ws=0), 1), (dict(norm=FAKE + 2), 3),
    (dict(ws=FAKE + 8), 3), (dict(wsb=16), 5), (dict(count=-1), 2),
    (dict(rows=[_row(p=0)]), 1), (dict(rows=[_row(p=FAKE + 1)]), 3), (dict(rows=[_row(n=-1)]), 2),
    (dict(rows=[_row(n=1 << 35)]), 2), (dict(rows=[_row(it=3, ot=3)]), 4),
])
def test_both_calls_reject_without_launch(lib, kw, status):
    assert _clip(lib, **kw) == status
    assert _clip(lib, clip=False, **kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(p=0), 1), (dict(p=FAKE + 1), 3), (dict(it=5), 4), (dict(size=(1, 1, -1, 5)), 2), (dict(si=(0, 0, -8, 1)), 2),
    (dict(size=(1 << 20, 1 << 20, 1, 1)), 2),
])
def test_strided_descriptors_are_checked(lib, kw, status):
    assert _clip(lib, strided=_strided(**kw)) == status
    assert _clip(lib, strided=_strided(**kw), clip=False) == status


@pytest.mark.parametrize("kw,status", [
    (dict(max_norm=-1.0), 4), (dict(max_norm=math.nan), 4), (dict(eps=-1.0), 4), (dict(eps=math.inf), 4),
    (dict(rows=[_row(q=0)]), 1), (dict(rows=[_row(q=FAKE + 1)]), 3), (dict(rows=[_row(ot=9)]), 4),
    (dict(rows=[_row(it=F32, ot=BF16)]), 4),                                  # in place with two types
    (dict(rows=[_row(), _row()]), 4),                                         # the same tensor twice
    (dict(rows=[_row(n=100), _row(p=FAKE + 198)]), 4),                        # the second starts inside the first
    (dict(rows=[_row(q=FAKE + 4096), _row(p=FAKE + 4100, q=FAKE + 8192)]), 4),  # an output over another's input
    (dict(rows=[_row(q=FAKE + 2)]), 4),                                       # an output one element further
    (dict(rows=[_row(q=FAKE + 4096, n=100, ot=F32), _row(p=FAKE + 400, q=FAKE + 4096 + 399 // 4 * 4, ot=F32)]), 4),
])
def test_clip_rejects_without_launch(lib, kw, status):
    assert _clip(lib, **kw) == status


@pytest.mark.skipif(torch.cuda.is_available(), reason="would launch on fake pointers when a GPU is present")
def test_valid_arguments_without_gpu_report_cuda_error(lib):
    neighbours = [_row(n=100), _row(p=FAKE + 200, n=0), _row(p=FAKE + 200, q=FAKE + 4096, n=3, ot=F32)]
    shared = [_row(q=FAKE + 4096), _row(q=FAKE + 8192)]  # one input into two outputs
    for rows in ([_row()], neighbours, shared, []):
        assert _clip(lib, rows=rows) in (6, 7)
        assert _clip(lib, rows=rows, clip=False) in (6, 7)
    assert _clip(lib, max_norm=math.inf) in (6, 7)
    assert _clip(lib, strided=_strided()) in (6, 7)
    assert _clip(lib, rows=[_row(), _row()], clip=False) in (6, 7)  # only read


def test_binding_refuses(lib):
    import linear_cross_entropy_gb300 as cce
    g = [torch.zeros(4)]
    for call in (lambda: cce.cce_grad_norm(g), lambda: cce.cce_clip_grads(g, 1.0)):
        with pytest.raises(ValueError, match="CUDA"):
            call()
    p = torch.zeros(4, requires_grad=True)
    p.grad = torch.ones(4)
    with pytest.raises(ValueError, match="CUDA"):
        cce.clip_grad_norm_(p, 1.0)
    with pytest.raises(ValueError, match="norm_type"):
        cce.cce_grad_norm(g, 3.0)
    with pytest.raises(ValueError, match="max_norm"):
        cce.cce_clip_grads(g, -1.0)
    with pytest.raises(ValueError, match="max_norm"):
        cce.cce_clip_grads(g, math.nan)
    with pytest.raises(ValueError, match="one tensor for each"):
        cce.cce_clip_grads(g, 1.0, out=[])


def test_no_gradients_is_a_norm_of_zero(lib):
    import linear_cross_entropy_gb300 as cce
    p = torch.zeros(4, requires_grad=True)
    assert cce.clip_grad_norm_([p], 1.0).item() == 0.0
    assert cce.cce_grad_norm([]).item() == 0.0
    assert cce.clip_grad_norm_(iter([p]), 1.0, error_if_nonfinite=True).item() == 0.0


def test_dimensions_of_strided_tensors(lib):
    from linear_cross_entropy_gb300.grads import _dims
    base = torch.zeros(6, 8, 10)
    assert _dims(base, base) == [(480, 1, 1)]
    t = base.transpose(0, 2)
    assert _dims(t, t) == [(480, 1, 1)]
    cut = base[:, :, 2:5]
    assert _dims(cut, cut) == [(48, 10, 10), (3, 1, 1)]
    assert _dims(cut, torch.empty(cut.shape)) == [(48, 10, 3), (3, 1, 1)]
    assert _dims(t, torch.empty(t.shape)) == [(10, 1, 48), (8, 10, 6), (6, 80, 1)]
    assert _dims(base[0, 0, :1], base[0, 0, :1]) == []
