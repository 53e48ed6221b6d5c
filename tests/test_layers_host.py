"""Host side of the linear and gated linear layers without a GPU: exported
symbols, workspaces, refusals of the C ABI before any launch and of the binding."""
import os
import re

import pytest
import torch
import torch.autograd.forward_ad as fwAD
from torch.fx.experimental.proxy_tensor import make_fx

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 1 << 20  # an aligned non-null host integer: never dereferenced, checks fail first
F32, F16, BF16, KEPT = 0, 1, 2, 3
NONE, RELU, GELU, GELU_TANH, SILU = range(5)


@pytest.fixture(scope="module")
def lib():
    from tests.conftest import build_library
    build_library()
    from linear_cross_entropy_gb300 import _lib
    return _lib.load()


@pytest.fixture(scope="module")
def cce(lib):
    import linear_cross_entropy_gb300
    return linear_cross_entropy_gb300


def test_declared_symbols(lib):
    src = open(os.path.join(ROOT, "include", "cce_layers.h")).read()
    names = set(re.findall(r"\b(cce_[a-z0-9_]+)\s*\(", re.sub(r"/\*.*?\*/", "", src, flags=re.S)))
    assert len(names) == 11 and all(hasattr(lib, n) for n in names)
    assert lib.cce_layers_abi_version() == 100


def _linear(lib, **kw):
    a = dict(x=FAKE, xp=64, w=FAKE, wp=64, type=BF16, b=FAKE, bt=F32, r=FAKE, ri=32, rp=100, ro=0, act=GELU, M=32, N=100,
             K=64, y=FAKE, yp=100, yt=BF16, z=FAKE, zp=100, zt=BF16, ws=FAKE, wsb=1 << 40)
    assert kw.keys() <= a.keys()
    return lib.cce_linear_forward(*(a | kw).values(), 0)


def _linear_backward(lib, **kw):
    a = dict(g=FAKE, gp=100, yt=BF16, x=FAKE, xp=64, w=FAKE, wp=64, type=BF16, z=FAKE, zp=100, zt=KEPT, act=GELU, M=32,
             N=100, K=64, dx=FAKE, dw=FAKE, db=FAKE, bt=F32, ws=FAKE, wsb=1 << 40)
    assert kw.keys() <= a.keys()
    return lib.cce_linear_backward(*(a | kw).values(), 0)


def _gated(lib, **kw):
    a = dict(x=FAKE, xp=64, w=FAKE, wp=64, u=FAKE, up=64, type=BF16, act=SILU, M=32, N=100, K=64, y=FAKE, yp=100,
             gate=FAKE, z=FAKE, zp=100, zt=KEPT, ws=FAKE, wsb=1 << 40)
    assert kw.keys() <= a.keys()
    return lib.cce_gated_linear_forward(*(a | kw).values(), 0)


def _gated_backward(lib, **kw):
    a = dict(g=FAKE, gp=100, x=FAKE, xp=64, w=FAKE, wp=64, u=FAKE, up=64, type=BF16, gate=FAKE, gatep=100, z=FAKE,
             zp=100, zt=BF16, act=SILU, M=32, N=100, K=64, dx=FAKE, dw=FAKE, du=FAKE, ws=FAKE, wsb=1 << 40)
    assert kw.keys() <= a.keys()
    return lib.cce_gated_linear_backward(*(a | kw).values(), 0)


CALLS = (_linear, _linear_backward, _gated, _gated_backward)


@pytest.mark.parametrize("kw,status", [
    (dict(zt=F16), 4), (dict(zt=F32), 4), (dict(type=F16, yt=F16, zt=KEPT), 4), (dict(zt=9), 4),
    (dict(x=0), 1), (dict(w=0), 1), (dict(type=F32), 4), (dict(type=7), 4), (dict(act=5), 4),
    (dict(act=-1), 4), (dict(M=-1), 2), (dict(N=0), 2), (dict(K=0), 2), (dict(M=1 << 31), 2), (dict(N=1 << 31), 2),
    (dict(M=(1 << 31) - 600, K=(1 << 31) - 600, xp=(1 << 31) - 8), 2), (dict(xp=56), 2), (dict(wp=56), 2),
    (dict(xp=1 << 31), 2), (dict(N=1 << 30, wp=1 << 30), 2), (dict(K=1 << 30, xp=1 << 30, wp=1 << 30), 2), (dict(xp=68), 3), (dict(wp=70), 3), (dict(x=FAKE + 8), 3), (dict(w=FAKE + 2), 3),
])
def test_every_call_rejects_without_launch(lib, kw, status):
    for call in CALLS:
        given = {k: v for k, v in kw.items() if k != "yt" or call in (_linear, _linear_backward)}
        assert call(lib, **given) == status, call


@pytest.mark.parametrize("kw,status", [(dict(ws=FAKE + 16), 3), (dict(wsb=8), 5), (dict(ws=0), 1)])
def test_workspaces_are_checked_where_one_is_needed(lib, kw, status):
    sizes = dict(M=100, N=600, K=9000, xp=9000, wp=9000)
    pitches = {_linear: ("rp", "yp", "zp"), _linear_backward: ("gp", "zp"), _gated: ("yp", "zp"),
               _gated_backward: ("gp", "zp", "gatep")}
    for call in CALLS:
        up = dict(up=9000) if call in (_gated, _gated_backward) else {}
        assert call(lib, **sizes, **{k: 600 for k in pitches[call]}, **up, **kw) == status, call


@pytest.mark.parametrize("kw,status", [
    (dict(bt=3), 4), (dict(yt=F16), 4), (dict(yt=5), 4), (dict(y=0), 1), (dict(rp=-1), 2), (dict(ri=0), 2), (dict(ro=-1), 2),
    (dict(ro=1 << 45), 2), (dict(yp=99), 2),
    (dict(rp=1 << 30), 2), (dict(yp=1 << 30), 2), (dict(zp=99), 2), (dict(b=FAKE + 2), 3), (dict(r=FAKE + 1), 3), (dict(y=FAKE + 1), 3), (dict(z=FAKE + 1), 3),
    (dict(yt=F32, y=FAKE + 2), 3), (dict(yt=F32, r=FAKE + 2), 3),
])
def test_linear_forward_rejects(lib, kw, status):
    assert _linear(lib, **kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(bt=3), 4), (dict(yt=F16), 4), (dict(g=0), 1), (dict(z=0), 1), (dict(gp=99), 2), (dict(zp=99), 2),
    (dict(g=FAKE + 1), 3), (dict(dx=FAKE + 1), 3), (dict(dw=FAKE + 1), 3), (dict(db=FAKE + 2), 3),
])
def test_linear_backward_rejects(lib, kw, status):
    assert _linear_backward(lib, **kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(u=0), 1), (dict(up=56), 2), (dict(up=65), 3), (dict(u=FAKE + 4), 3), (dict(y=0), 1), (dict(gate=0), 1),
    (dict(z=0), 1), (dict(zp=99), 2), (dict(yp=99), 2), (dict(y=FAKE + 1), 3), (dict(gate=FAKE + 1), 3),
])
def test_gated_forward_rejects(lib, kw, status):
    assert _gated(lib, **kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(u=0), 1), (dict(g=0), 1), (dict(gate=0), 1), (dict(z=0), 1), (dict(gp=99), 2), (dict(gatep=99), 2),
    (dict(du=FAKE + 1), 3),
])
def test_gated_backward_rejects(lib, kw, status):
    assert _gated_backward(lib, **kw) == status


@pytest.mark.skipif(torch.cuda.is_available(), reason="would launch on fake pointers when a GPU is present")
def test_valid_arguments_without_gpu_report_cuda_error(lib):
    for call in CALLS:
        assert call(lib) in (6, 7)
        assert call(lib, M=0) in (6, 7)
        assert call(lib, M=1) in (6, 7)
    assert _linear(lib, b=0, r=0, z=0) in (6, 7) and _linear(lib, yt=F32) in (6, 7)
    assert _linear_backward(lib, act=NONE, z=0) in (6, 7)
    assert _linear_backward(lib, dx=0, dw=0, db=0) in (6, 7)
    assert _gated(lib, gate=0, z=0) in (6, 7)
    from linear_cross_entropy_gb300._lib import RowCopy
    assert lib.cce_copy_rows((RowCopy * 1)(RowCopy(FAKE, 2 * FAKE, 3, 100, 400, 104, 9, 100, 2)), 1, 0) in (6, 7)
    assert _linear(lib, M=16, ws=0, wsb=0) in (6, 7)  # few rows need no workspace


@pytest.mark.parametrize("kw,status", [
    (dict(src=0), 1), (dict(dst=0), 1), (dict(inner=0), 2), (dict(row_stride=-1), 2), (dict(outer_stride=-1), 2),
    (dict(pitch=99), 2), (dict(pitch=108), 3), (dict(rows=-1), 2), (dict(cols=-1), 2), (dict(rows=1 << 31), 2),
    (dict(bytes=8), 4), (dict(src=FAKE + 1), 3), (dict(dst=FAKE + 8), 3), (dict(bytes=4, src=FAKE + 2), 3),
])
def test_row_copies_are_checked(lib, kw, status):
    from linear_cross_entropy_gb300._lib import RowCopy
    a = dict(src=FAKE, dst=2 * FAKE, inner=3, row_stride=100, outer_stride=400, pitch=104, rows=9, cols=100, bytes=2)
    good, bad = RowCopy(*a.values()), RowCopy(*(a | kw).values())
    assert lib.cce_copy_rows((RowCopy * 2)(good, bad), 2, 0) == status
    assert lib.cce_copy_rows(None, 1, 0) == 1 and lib.cce_copy_rows((RowCopy * 1)(good), -1, 0) == 4
    assert lib.cce_copy_rows((RowCopy * 9)(*[good] * 9), 9, 0) == 4


def test_workspaces(cce):
    q = (cce.linear_forward_workspace_bytes, cce.linear_backward_workspace_bytes,
         cce.gated_linear_forward_workspace_bytes, cce.gated_linear_backward_workspace_bytes)
    for f in q:
        assert f(-1, 8, 8) == f(8, 0, 8) == f(8, 8, 0) == f(1 << 31, 8, 8) == f(1 << 30, 1 << 30, 8) == 0
        for M, N, K in [(0, 8, 8), (1, 1, 1), (16, 4096, 4096), (17, 70000, 16), (4096, 896, 896), (65536, 2048, 8192)]:
            # what is staged of dz, sums of a bias and at most 256 MiB of partial sums for each product
            b = f(M, N, K)
            assert 16 <= b <= 4 * (M + 1) * (N + 8) + 1024 * N + (3 << 28) + 4096, (f, M, N, K)
    assert cce.linear_forward_workspace_bytes(16, 4096, 4096) == 16  # few rows need none
    assert cce.linear_backward_workspace_bytes(100, 24, 8) >= 2 * 100 * 24


def test_binding_refuses(cce):
    x, w = torch.zeros(4, 8, dtype=torch.bfloat16), torch.zeros(3, 8, dtype=torch.bfloat16)
    y = torch.zeros(4, 3, dtype=torch.bfloat16)
    for call in (lambda: cce.linear(x, w), lambda: cce.cce_linear_forward(x, w), lambda: cce.gated_linear(x, w, w),
                 lambda: cce.cce_linear_backward(y, x, w), lambda: cce.cce_gated_linear_forward(x, w, w),
                 lambda: cce.cce_gated_linear_backward(y, x, w, w, y, y)):
        with pytest.raises(ValueError, match="CUDA"):
            call()


def test_tangents_and_tracing_are_refused(cce):
    x, w = torch.zeros(4, 8), torch.zeros(3, 8)
    y = torch.zeros(4, 3)
    with fwAD.dual_level():
        d, dw, dy = (fwAD.make_dual(t, torch.ones_like(t)) for t in (x, w, y))
        for call in (lambda: cce.linear(d, w), lambda: cce.linear(x, dw), lambda: cce.linear(x, w, dy[0]),
                     lambda: cce.linear(x, w, residual=dy), lambda: cce.gated_linear(d, w, w),
                     lambda: cce.gated_linear(x, w, dw), lambda: cce.cce_linear_backward(dy, x, w),
                     lambda: cce.cce_linear_backward(y, x, w, dy, "gelu"),
                     lambda: cce.cce_gated_linear_backward(y, x, w, w, y, dy)):
            with pytest.raises(NotImplementedError, match="tangent"):
                call()
    for call in (lambda x: cce.linear(x, w), lambda x: cce.gated_linear(x, w, w),
                 lambda x: cce.cce_linear_backward(y, x, w)[0],
                 lambda x: cce.cce_gated_linear_backward(y, x, w, w, y, y)[0]):
        with pytest.raises(NotImplementedError, match="traced"):
            torch.jit.trace(call, (x,))
        with pytest.raises(NotImplementedError, match="traced"):
            make_fx(call)(x)


def test_no_errors_are_pending_without_a_gpu(cce):
    cce.raise_pending_errors()
