"""What the statuses' texts say holds for both headers."""
import pytest


@pytest.fixture(scope="module")
def lib():
    from tests.conftest import build_library
    build_library()
    from linear_cross_entropy_gb300 import _lib
    return _lib.load()


@pytest.mark.parametrize("status,words", [(2, "stride"), (3, "element"), (4, "overlap")])
def test_texts_fit_the_operators_around_the_head(lib, status, words):
    assert words in lib.cce_status_string(status).decode()
