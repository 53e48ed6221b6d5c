"""Forward-mode derivatives and tracing, which pass a call of the norms or of
clipping by, are refused, and not answered with a tangent of 0 or a graph that
holds an empty tensor."""
import pytest
import torch
import torch.autograd.forward_ad as fwAD
from torch._subclasses.fake_tensor import FakeTensorMode
from torch.fx.experimental.proxy_tensor import make_fx


@pytest.fixture(scope="module")
def cce():
    from tests.conftest import build_library
    build_library()
    import linear_cross_entropy_gb300
    return linear_cross_entropy_gb300


def _calls(cce, x, w, g):
    """Every call, with the argument that is not plain in each place in turn."""
    plain_x, plain_w, stat = torch.zeros(4, 8), torch.zeros(8), torch.zeros(4)
    return [lambda: cce.layer_norm(x), lambda: cce.layer_norm(plain_x, w), lambda: cce.layer_norm(plain_x, plain_w, w),
            lambda: cce.rms_norm(x, plain_w), lambda: cce.rms_norm(plain_x, w),
            lambda: cce.cce_layer_norm_forward(x, plain_w), lambda: cce.cce_rms_norm_forward(x),
            lambda: cce.cce_layer_norm_backward(plain_x, x, plain_w, stat, stat),
            lambda: cce.cce_rms_norm_backward(plain_x, plain_x, w, stat),
            lambda: cce.cce_grad_norm([plain_x, g]), lambda: cce.cce_clip_grads([g], 1.0),
            lambda: cce.cce_clip_grads([plain_x], 1.0, out=[g])]


def test_tangents_are_refused(cce):
    with fwAD.dual_level():
        x, w, g = (fwAD.make_dual(torch.zeros(s), torch.ones(s)) for s in ((4, 8), (8,), (4, 8)))
        for i, call in enumerate(_calls(cce, x, w, g)):
            # the plain gradient ahead of the dual one is refused for its device first
            with pytest.raises((NotImplementedError, ValueError) if i == 9 else NotImplementedError):
                call()
        with torch.no_grad(), pytest.raises(NotImplementedError, match="tangent"):
            cce.layer_norm(x, w)
        with pytest.raises(NotImplementedError, match="tangent"):
            cce.rms_norm(x.clone().requires_grad_(), w)
        # tensors without a tangent are as before
        with pytest.raises(ValueError, match="CUDA"):
            cce.layer_norm(torch.zeros(4, 8))
    with pytest.raises(NotImplementedError, match="tangent"):
        torch.func.jvp(cce.rms_norm, (torch.zeros(4, 8),), (torch.ones(4, 8),))


def test_tracing_is_refused(cce):
    x, w = torch.zeros(4, 8), torch.ones(8)
    calls = [lambda x: cce.layer_norm(x, w), lambda x: cce.rms_norm(x), lambda x: cce.cce_rms_norm_forward(x, w)[0],
             lambda x: cce.cce_layer_norm_backward(x, x, w, x[:, 0], x[:, 0])[0],
             lambda x: cce.cce_grad_norm([x]), lambda x: cce.cce_clip_grads([x], 1.0)]
    for call in calls:
        with pytest.raises(NotImplementedError, match="traced"):
            torch.jit.trace(call, (x,))
        for mode in ("real", "fake", "symbolic"):
            with pytest.raises(NotImplementedError, match="traced"):
                make_fx(call, tracing_mode=mode)(x)


@pytest.mark.skipif(torch.cuda.is_available(), reason="fake CUDA tensors need no GPU; a real one is not touched")
def test_fake_tensors_give_no_result(cce):
    with FakeTensorMode():
        x, w = torch.empty(4, 8, device="cuda"), torch.empty(8, device="cuda")
        for call in (lambda: cce.layer_norm(x, w), lambda: cce.rms_norm(x), lambda: cce.cce_grad_norm([x])):
            with pytest.raises(RuntimeError):
                call()
