"""Workspaces of the layers' backward calls without a GPU: a call needs what it computes, and no more."""
import itertools

import pytest
import torch

from tests import test_layers_host as H

DX, DW, DW_UP, DB, DZ = 1, 2, 4, 8, 16
SIZES = [(1, 1, 1), (17, 70000, 16), (100, 600, 9000), (4096, 896, 896), (4096, 152, 70000), (65536, 8192, 2048), (64, 151936, 896)]


@pytest.fixture(scope="module")
def lib():
    from tests.conftest import build_library
    build_library()
    from linear_cross_entropy_gb300 import _lib
    return _lib.load()


@pytest.mark.parametrize("M,N,K", SIZES)
def test_no_call_needs_more_than_any(lib, M, N, K):
    for flags in itertools.product(*((0, f) for f in (DX, DW, DB, DZ))):
        assert 16 <= lib.cce_linear_backward_workspace_bytes_ex(M, N, K, sum(flags)) <= lib.cce_linear_backward_workspace_bytes(M, N, K)
    for flags in itertools.product(*((0, f) for f in (DX, DW, DW_UP))):
        assert 16 <= lib.cce_gated_linear_backward_workspace_bytes_ex(M, N, K, sum(flags)) <= \
            lib.cce_gated_linear_backward_workspace_bytes(M, N, K)
    assert lib.cce_linear_backward_workspace_bytes_ex(M, N, K, 0) == lib.cce_gated_linear_backward_workspace_bytes_ex(M, N, K, 0) == 16


def test_what_is_not_computed_takes_nothing(lib):
    q = lib.cce_linear_backward_workspace_bytes_ex
    # a plain projection's gradients: no dz of its own (1 GiB), no sums of a bias
    assert q(65536, 8192, 2048, DX | DW) <= 2 << 28
    assert q(65536, 8192, 2048, DX | DW | DZ) >= 2 * 65536 * 8192
    # sums of a wide layer: six blocks an SM in all, 1,216 columns' worth and a row for each at least
    assert q(4096, 151936, 896, DB) <= 4 * 2 * 151936 + 256
    assert q(4096, 896, 896, DB) <= 4 * 256 * 896 + 256


def test_invalid_ones(lib):
    for q, bad in ((lib.cce_linear_backward_workspace_bytes_ex, DW_UP), (lib.cce_gated_linear_backward_workspace_bytes_ex, DB)):
        assert q(-1, 8, 8, DX) == q(8, 0, 8, DX) == q(8, 8, 0, DX) == q(1 << 31, 8, 8, DX) == 0
        assert q(8, 8, 8, bad) == q(8, 8, 8, 32) == q(8, 8, 8, -1) == 0
        assert q(0, 8, 8, DX | DW) == 16


@pytest.mark.skipif(torch.cuda.is_available(), reason="would launch on fake pointers when a GPU is present")
def test_a_call_asks_for_no_more(lib):
    M, N, K = 100, 600, 9000
    at = dict(M=M, N=N, K=K, xp=K, wp=K, gp=N, zp=N)
    for dx, dw, db, act in itertools.product((0, 1), (0, 1), (0, 1), (H.NONE, H.GELU)):
        staged = DZ if act != H.NONE and (dx or dw) else 0
        need = lib.cce_linear_backward_workspace_bytes_ex(M, N, K, DX * dx | DW * dw | DB * db | staged)
        call = dict(at, act=act, dx=H.FAKE * dx, dw=H.FAKE * dw, db=H.FAKE * db)
        assert H._linear_backward(lib, **call, wsb=need) in (6, 7)
        if need > 16:
            assert H._linear_backward(lib, **call, wsb=need - 1) == 5
    # grad_y that the products cannot read
    for other in (dict(g=H.FAKE + 2), dict(gp=N + 1), dict(yt=H.F32)):
        call = dict(at, act=H.NONE, db=0) | other
        need = lib.cce_linear_backward_workspace_bytes_ex(M, N, K, DX | DW | DZ)
        assert H._linear_backward(lib, **call, wsb=need) in (6, 7) and H._linear_backward(lib, **call, wsb=need - 1) == 5
    for dx, dw, du in itertools.product((0, 1), repeat=3):
        need = lib.cce_gated_linear_backward_workspace_bytes_ex(M, N, K, DX * dx | DW * dw | DW_UP * du)
        call = dict(at, up=K, gatep=N, dx=H.FAKE * dx, dw=H.FAKE * dw, du=H.FAKE * du)
        assert H._gated_backward(lib, **call, wsb=need) in (6, 7)
        if need > 16:
            assert H._gated_backward(lib, **call, wsb=need - 1) == 5
