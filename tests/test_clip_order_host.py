"""An output that starts where its input does but orders the elements otherwise is
refused before any launch: threads would write what others have yet to read."""
import ctypes

import pytest
import torch

FAKE = 1 << 20  # an aligned non-null host integer: never dereferenced, checks fail first
SIX_SEVEN = (6, 7)  # no GPU: the checks of the arguments have passed


@pytest.fixture(scope="module")
def lib():
    from tests.conftest import build_library
    build_library()
    from linear_cross_entropy_gb300 import _lib
    return _lib.load()


def _status(lib, size, si, so, out=FAKE, clip=True):
    from linear_cross_entropy_gb300._lib import Strided
    four = ctypes.c_int64 * 4
    s = (Strided * 1)(Strided(FAKE, out, 0, 0, four(*size), four(*si), four(*so)))
    args = (0, 0, ctypes.addressof(s), 1, 2)
    if clip:
        return lib.cce_clip_grads(*args, 1.0, 1e-6, FAKE, FAKE, 1 << 30, 0)
    return lib.cce_grad_norm(*args, FAKE, FAKE, 1 << 30, 0)


@pytest.mark.parametrize("size,si,so", [((1, 1, 8, 8), (0, 0, 8, 1), (0, 0, 1, 8)), ((1, 1, 3, 5), (0, 0, 8, 1), (0, 0, 5, 1)),
                                        ((2, 1, 3, 5), (40, 0, 8, 1), (80, 0, 8, 1))])
def test_another_order_in_place_is_refused(lib, size, si, so):
    assert _status(lib, size, si, so) == 4


@pytest.mark.skipif(torch.cuda.is_available(), reason="would launch on fake pointers when a GPU is present")
def test_the_same_order_and_other_memory_are_not(lib):
    cut = ((1, 1, 3, 5), (0, 0, 8, 1))
    assert _status(lib, *cut, (0, 0, 8, 1)) in SIX_SEVEN
    assert _status(lib, *cut, (7, 9, 8, 1)) in SIX_SEVEN  # strides of dimensions of size 1 say nothing
    assert _status(lib, *cut, (0, 0, 5, 1), out=FAKE + 4096) in SIX_SEVEN
    assert _status(lib, *cut, (0, 0, 5, 1), clip=False) in SIX_SEVEN  # outputs are not read
