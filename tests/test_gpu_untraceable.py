"""Forward-mode derivatives and traced graphs of the norms and of clipping are
refused on the GPU, where a call would otherwise run; beside them plain tensors
go through."""
import pytest
import torch
import torch.autograd.forward_ad as fwAD
from torch.fx.experimental.proxy_tensor import make_fx

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def cce():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    from tests.conftest import build_library
    build_library()
    import linear_cross_entropy_gb300
    return linear_cross_entropy_gb300


def test_tangents(cce):
    x, w = torch.randn(4, 64, device="cuda"), torch.ones(64, device="cuda")
    want = cce.layer_norm(x, w)
    with fwAD.dual_level():
        dual = fwAD.make_dual(x.clone(), torch.ones_like(x))
        dual_w = fwAD.make_dual(w.clone(), torch.ones_like(w))
        for call in (lambda: cce.layer_norm(dual, w), lambda: cce.rms_norm(x, dual_w),
                     lambda: cce.layer_norm(x, w, dual_w), lambda: cce.cce_rms_norm_forward(dual, w),
                     lambda: cce.cce_rms_norm_backward(dual, x, w, x[:, 0].contiguous()),
                     lambda: cce.cce_grad_norm([x, dual]), lambda: cce.cce_clip_grads([dual], 1.0)):
            with pytest.raises(NotImplementedError, match="tangent"):
                call()
            with torch.no_grad(), pytest.raises(NotImplementedError, match="tangent"):
                call()
        assert torch.equal(cce.layer_norm(x, w), want)
    with pytest.raises(NotImplementedError, match="tangent"):
        torch.func.jvp(cce.rms_norm, (x,), (x,))


def test_traced_graphs(cce):
    x, w = torch.randn(4, 64, device="cuda"), torch.ones(64, device="cuda")
    for call in (lambda t: cce.layer_norm(t, w), lambda t: cce.rms_norm(t), lambda t: cce.cce_grad_norm([t])):
        with pytest.raises(NotImplementedError, match="traced"):
            torch.jit.trace(call, (x,))
        with pytest.raises(NotImplementedError, match="traced"):
            make_fx(call)(x)
        call(x)


def test_second_derivative_of_a_recorded_tangent(cce):
    """Forward over reverse: the backward's upstream gradient has a tangent."""
    x = torch.randn(4, 64, device="cuda", requires_grad=True)
    with fwAD.dual_level():
        y = cce.rms_norm(x)
        g = fwAD.make_dual(torch.ones_like(x), torch.ones_like(x))
        with pytest.raises(RuntimeError, match="tangent"):
            torch.autograd.grad(y, x, g)
