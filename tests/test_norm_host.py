"""Host side of the norms without a GPU: exports, workspace sizes, refusals
of the C ABI before any launch and of the Python binding, and how rows of
views are described."""
import ctypes
import os
import re

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def lib():
    from tests.conftest import build_library
    build_library()
    from linear_cross_entropy_gb300 import _lib
    return _lib.load()


def test_exports_every_declared_symbol(lib):
    src = open(os.path.join(ROOT, "include", "cce_ops.h")).read()
    src = re.sub(r"/\*.*?\*/", "", src, flags=re.S)
    names = sorted(set(re.findall(r"\b(cce_[a-z0-9_]+)\s*\(", src)))
    assert "cce_layer_norm_forward" in names
    for n in names:
        assert hasattr(lib, n), n
    assert lib.cce_ops_abi_version() == 100


def test_backward_workspace(lib):
    for N, D in [(1, 1), (1, 896), (4096, 896), (65536, 2048), (7, 100003)]:
        b = lib.cce_norm_backward_workspace_bytes(N, D)
        assert b >= 2 * 4 * D * min(N, 304)
        assert b <= 2 * (4 * D * min(N, 304) + 256)
    assert lib.cce_norm_backward_workspace_bytes(0, 8) > 0
    for N, D in [(-1, 8), (8, 0), (1 << 31, 8), (8, 1 << 31)]:
        assert lib.cce_norm_backward_workspace_bytes(N, D) == 0


FAKE = 1 << 20  # an aligned non-null host integer: never dereferenced, checks fail first
NAN, INF = float("nan"), float("inf")


def _forward(lib, layer, **kw):
    a = dict(x=FAKE, inner=8, row=64, outer=0, xt=2, w=FAKE, b=FAKE, pt=2, off=0.0, N=8, D=64, eps=1e-5, y=FAKE, yt=2,
             mean=FAKE, rstd=FAKE)
    a.update(kw)
    head = (a["x"], a["inner"], a["row"], a["outer"], a["xt"], a["w"])
    if layer:
        return lib.cce_layer_norm_forward(*head, a["b"], a["pt"], a["N"], a["D"], a["eps"], a["y"], a["yt"], a["mean"],
                                          a["rstd"], 0)
    return lib.cce_rms_norm_forward(*head, a["pt"], a["off"], a["N"], a["D"], a["eps"], a["y"], a["yt"], a["rstd"], 0)


def _backward(lib, layer, **kw):
    a = dict(g=FAKE, gi=8, gr=64, go=0, yt=2, x=FAKE, xi=8, xr=64, xo=0, xt=2, w=FAKE, pt=2, off=0.0, mean=FAKE,
             rstd=FAKE, N=8, D=64, dx=FAKE, dw=FAKE, db=FAKE, ws=FAKE, wsb=1 << 30)
    a.update(kw)
    head = (a["g"], a["gi"], a["gr"], a["go"], a["yt"], a["x"], a["xi"], a["xr"], a["xo"], a["xt"], a["w"], a["pt"])
    if layer:
        return lib.cce_layer_norm_backward(*head, a["mean"], a["rstd"], a["N"], a["D"], a["dx"], a["dw"], a["db"],
                                           a["ws"], a["wsb"], 0)
    return lib.cce_rms_norm_backward(*head, a["off"], a["rstd"], a["N"], a["D"], a["dx"], a["dw"], a["ws"], a["wsb"],
                                     0)


@pytest.mark.parametrize("layer", [True, False])
@pytest.mark.parametrize("kw,status", [
    (dict(x=0), 1), (dict(y=0), 1),
    (dict(N=-1), 2), (dict(N=1 << 31), 2), (dict(D=0), 2), (dict(D=1 << 31), 2), (dict(inner=0), 2),
    (dict(row=-1), 2), (dict(outer=-8), 2),
    (dict(x=FAKE + 1), 3), (dict(y=FAKE + 1), 3), (dict(w=FAKE + 1), 3), (dict(rstd=FAKE + 2), 3),
    (dict(xt=3), 4), (dict(yt=-1), 4), (dict(pt=7), 4), (dict(xt=2, yt=1), 4), (dict(xt=2, yt=0), 4),
    (dict(eps=-1.0), 4), (dict(eps=NAN), 4), (dict(eps=INF), 4),
])
def test_forward_rejects_without_launch(lib, layer, kw, status):
    assert _forward(lib, layer, **kw) == status


@pytest.mark.parametrize("layer", [True, False])
@pytest.mark.parametrize("kw,status", [
    (dict(g=0), 1), (dict(x=0), 1), (dict(rstd=0), 1), (dict(ws=0), 1),
    (dict(N=-1), 2), (dict(D=0), 2), (dict(gi=0), 2), (dict(gr=-1), 2), (dict(xo=-1), 2),
    (dict(g=FAKE + 1), 3), (dict(x=FAKE + 1), 3), (dict(dx=FAKE + 1), 3), (dict(dw=FAKE + 1), 3),
    (dict(ws=FAKE + 8), 3),
    (dict(yt=1), 4), (dict(yt=0), 4), (dict(pt=3), 4), (dict(wsb=100), 5),
])
def test_backward_rejects_without_launch(lib, layer, kw, status):
    assert _backward(lib, layer, **kw) == status


def test_layer_only_arguments(lib):
    assert _forward(lib, True, b=FAKE + 1) == 3
    assert _forward(lib, True, mean=FAKE + 2) == 3
    assert _forward(lib, False, off=NAN) == 4
    assert _backward(lib, True, mean=0) == 1
    assert _backward(lib, True, db=FAKE + 1) == 3
    assert _backward(lib, False, off=INF) == 4


@pytest.mark.skipif(torch.cuda.is_available(), reason="would launch on fake pointers when a GPU is present")
def test_valid_arguments_without_gpu_report_cuda_error(lib):
    for layer in (True, False):
        assert _forward(lib, layer) in (6, 7)
        assert _backward(lib, layer) in (6, 7)


def test_binding_refuses_cpu_tensors_and_bad_shapes(lib):
    import linear_cross_entropy_gb300 as cce
    x, w = torch.zeros(4, 8), torch.zeros(8)
    for call in (lambda: cce.layer_norm(x, w), lambda: cce.rms_norm(x, w), lambda: cce.layer_norm(x),
                 lambda: cce.cce_layer_norm_backward(x, x, w, x[:, 0], x[:, 0]),
                 lambda: cce.cce_rms_norm_backward(x, x, w, x[:, 0])):
        with pytest.raises(ValueError, match="CUDA"):
            call()


def test_rows_of_views(lib):
    """Views whose rows lie at one pitch, or in runs at one pitch, are read in
    place; the description addresses the view's own elements."""
    from linear_cross_entropy_gb300.norm import _rows
    base = torch.arange(5 * 6 * 8 * 2, dtype=torch.float32)
    full = base.view(5, 6, 16)
    views = [full, full[:, :-1], full[:, 1:], full[..., :8], full[::2], full[:, 0], full[0, 0], full[:, ::2, 4:12],
             full[:1, :3], full[2:3, 1:2], full.transpose(0, 1), full[0, 0].expand(7, 16), full[:, :0],
             base.view(5, 2, 3, 16)[:, :, :2][:, :1], base.as_strided((3, 4), (1, 1)), full[..., :1]]
    for v in views:
        t, inner, row, outer = _rows(v)
        assert t.data_ptr() == v.data_ptr()
        want = v.reshape(-1, v.shape[-1])
        for n in range(want.shape[0]):
            at = t.storage_offset() + n // inner * outer + n % inner * row
            assert torch.equal(base[at:at + v.shape[-1]], want[n]), v.shape
    for v in (full[..., ::2], full.transpose(1, 2), base.view(5, 2, 3, 16)[:, :, :2][..., 1:3][:4].transpose(0, 2)):
        t, inner, row, outer = _rows(v)
        assert t.is_contiguous() and torch.equal(t, v) and (row, outer) == (v.shape[-1], 0)
