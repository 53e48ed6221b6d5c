"""Tile plans of the layers without a GPU: a repeated call searches none."""
import random

import pytest


@pytest.fixture(scope="module")
def lib():
    from tests.conftest import build_library
    build_library()
    from linear_cross_entropy_gb300 import _lib
    return _lib.load()


def queries(lib, M, N, K):
    return [getattr(lib, f"cce_{name}_workspace_bytes")(M, N, K)
            for name in ("linear_forward", "linear_backward", "gated_linear_forward", "gated_linear_backward")]


def test_a_repeated_call_searches_nothing(lib):
    rng = random.Random(1)
    shapes = [(4096, 4096, 4096), (2048, 11008, 4096), (64, 64, 64), (1, 1, 1)]
    shapes += [tuple(round(2 ** rng.uniform(6, 14)) for _ in range(3)) for _ in range(400)]
    for shape in shapes:
        first = queries(lib, *shape)
        before = lib.cce_layers_plan_searches()
        for _ in range(3):
            assert queries(lib, *shape) == first
        assert lib.cce_layers_plan_searches() == before, shape


def test_the_layers_of_a_model_keep_their_plans(lib):
    """Twenty layers of four operators each, all of their own sizes, one after another."""
    layers = [(2048 + 64 * i, 1024 + 128 * i, 896 + 64 * i) for i in range(20)]
    first = [queries(lib, *s) for s in layers]
    before = lib.cce_layers_plan_searches()
    assert [queries(lib, *s) for s in layers] == first
    assert lib.cce_layers_plan_searches() == before


def test_threads_share_them(lib):
    import threading
    queries(lib, 3000, 1111, 777)
    before = lib.cce_layers_plan_searches()
    got = []
    threads = [threading.Thread(target=lambda: got.append(queries(lib, 3000, 1111, 777))) for _ in range(8)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert all(g == got[0] for g in got) and lib.cce_layers_plan_searches() == before
