"""A wait of the layers' products that runs out, without a fault: it ends, its device's
error word is given once, and the context stays usable."""
import ctypes

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    from tests.conftest import build_library
    build_library()
    from linear_cross_entropy_gb300 import _lib
    return _lib.load()


def test_a_wait_that_runs_out_is_reported_once(lib):
    import linear_cross_entropy_gb300 as cce
    x, w = (torch.randn(n, 64, device="cuda").bfloat16() for n in (300, 72))
    want = cce.linear(x, w)
    cce.raise_pending_errors()
    stream = torch.cuda.current_stream().cuda_stream
    word = ctypes.c_int32(-1)
    assert lib.cce_selftest_layers_wait_timeout(20000, stream) == 0
    assert lib.cce_layers_take_error(ctypes.addressof(word), stream) == 0 and word.value == cce.DEVERR_TIMEOUT
    assert lib.cce_layers_take_error(ctypes.addressof(word), stream) == 0 and word.value == 0
    assert lib.cce_selftest_layers_wait_timeout(20000, stream) == 0
    with pytest.raises(cce.CCEError, match="TIMEOUT"):
        cce.raise_pending_errors()
    cce.raise_pending_errors()
    assert torch.equal(cce.linear(x, w), want)


def test_its_limit_is_checked(lib):
    assert lib.cce_selftest_layers_wait_timeout(0, 0) == lib.cce_selftest_layers_wait_timeout(10000001, 0) == 4
