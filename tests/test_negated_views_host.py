"""Views that torch negates lazily (the imaginary part of a conjugate) are read as
the values that they stand for; the memory holds the others."""
import pytest
import torch


@pytest.fixture(scope="module")
def native():
    from tests.conftest import build_library
    build_library()
    import linear_cross_entropy_gb300  # noqa: F401  (loads what the module links against)
    from linear_cross_entropy_gb300 import _native
    return _native


def test_rows_are_the_values(native):
    base = torch.arange(24.0).view(4, 6)
    for view in (torch._neg_view(base), torch._neg_view(base)[:, :5], torch.complex(base, base).conj().imag):
        assert view.is_neg()
        rows = native.rows(view)[0]
        assert not rows.is_neg() and torch.equal(rows, view)
    assert native.rows(base)[0].data_ptr() == base.data_ptr()
