"""The norms and clipping on views that torch negates lazily."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def cce():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    from tests.conftest import build_library
    build_library()
    import linear_cross_entropy_gb300
    return linear_cross_entropy_gb300


def test_norms(cce):
    x, dy = torch.randn(2, 7, 136, device="cuda").unbind()
    w, b = torch.randn(2, 136, device="cuda").unbind()
    views = [torch._neg_view(t) for t in (x, w, b, dy)]
    values = [v.resolve_neg() for v in views]
    (x, w, b, dy), (x2, w2, b2, dy2) = views, values
    got, want = cce.cce_layer_norm_forward(x, w, b), cce.cce_layer_norm_forward(x2, w2, b2)
    grads = cce.cce_layer_norm_backward(dy, x, w, *got[1:]), cce.cce_layer_norm_backward(dy2, x2, w2, *want[1:])
    rms = cce.cce_rms_norm_forward(x, w), cce.cce_rms_norm_forward(x2, w2)
    rms_grads = cce.cce_rms_norm_backward(dy, x, w, rms[0][1]), cce.cce_rms_norm_backward(dy2, x2, w2, rms[1][1])
    for a, c in ((got, want), grads, rms, rms_grads, ((cce.layer_norm(x, w, b),), (cce.layer_norm(x2, w2, b2),))):
        assert all(torch.equal(s, t) for s, t in zip(a, c))
    with pytest.raises(ValueError, match="mean"):
        cce.cce_layer_norm_backward(dy, x, w, torch._neg_view(got[1]), got[2])


def test_clipping(cce):
    base = torch.randn(60, 80, device="cuda")
    for g in (torch._neg_view(base), torch.complex(base, base).conj().imag):
        assert g.is_neg()
        norm = cce.cce_grad_norm([g])
        want = g.resolve_neg().double().norm().item()
        assert abs(norm.item() - want) <= 2.0 ** -18 * want
        with pytest.raises(ValueError, match="negated"):
            cce.cce_clip_grads([g], 1.0, out=[torch.empty_like(base)])
        with pytest.raises(ValueError, match="negated"):
            cce.cce_clip_grads([torch.empty_like(base)], 1.0, out=[g])
        before = g.clone()
        cce.cce_clip_grads([g], 1.0)
        torch.testing.assert_close(g.resolve_neg(), before / (norm + 1e-6), rtol=2.0 ** -21, atol=0)
