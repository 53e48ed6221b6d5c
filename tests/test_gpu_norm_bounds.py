"""Layer norm and RMS norm with rows whose mean is far from 0, by the bounds of
tests/norm_bounds.py, on each kernel: rows in registers, in the cluster, spread
over blocks, shifted and beyond the registers."""
import numpy as np
import pytest
import torch

from tests import norm_bounds as B

pytestmark = pytest.mark.gpu

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def cce():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    from tests.conftest import build_library
    build_library()
    import linear_cross_entropy_gb300
    return linear_cross_entropy_gb300


def _d(t):
    return t.detach().double().cpu().numpy()


@pytest.mark.parametrize("layer", [True, False])
@pytest.mark.parametrize("mean", [0.0, 10.0, 1000.0])
@pytest.mark.parametrize("x_type,y_type", [(F32, F32), (F32, BF16), (F32, F16), (BF16, BF16)])
@pytest.mark.parametrize("N,D", [(1, 896), (2, 33), (3, 5), (6, 1001), (40, 4096), (700, 896), (650, 1001), (5, 9000),
                                 (4, 16392), (4, 30000), (3, 33000), (2, 33001)])
def test_rows_far_from_zero(cce, layer, mean, x_type, y_type, N, D):
    gen = torch.Generator(device="cuda").manual_seed(N * 101 + D)

    def randn(*shape):
        return torch.randn(shape, generator=gen, device="cuda")

    eps = 1e-5
    x, dy = (randn(N, D) + mean).to(x_type), randn(N, D).to(y_type)
    w, b = 1 + 0.3 * randn(D), 0.3 * randn(D)
    if layer:
        y, m, r = cce.cce_layer_norm_forward(x, w, b, eps, out_dtype=y_type)
        dx, dw, db = cce.cce_layer_norm_backward(dy, x, w, m, r)
    else:
        y, r = cce.cce_rms_norm_forward(x, w, eps, out_dtype=y_type)
        dx, dw = cce.cce_rms_norm_backward(dy, x, w, r)
    md = _d(m) if layer else np.zeros(N)
    rd, xd, wd, bd = _d(r), _d(x), _d(w), _d(b) if layer else np.zeros(D)
    assert B.stats_outside(md, rd, xd, eps, layer) == (0, 0)
    assert B.y_outside(_d(y), xd, wd, bd, md, rd, y_type) == 0
    assert B.grads_outside(_d(dx), _d(dw), _d(dy), xd, wd, md, rd, layer, x_type, F32) == (0, 0)
    if layer:
        g = _d(dy)
        assert B.outside(_d(db), g.sum(axis=0), B.depth(N) * B.u * np.abs(g).sum(axis=0), F32) == 0
