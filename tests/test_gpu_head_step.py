"""The head's training step on the GPU: norm, classifier with cross entropy,
backward pass and clipping together, against the same chain in 64 bits."""
import importlib.util
import os

import pytest
import torch

from tests.gpu_util import TOL_GRAD

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    from tests.conftest import build_library
    build_library()
    spec = importlib.util.spec_from_file_location("head_step", os.path.join(ROOT, "examples", "head_step.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


@pytest.mark.parametrize("norm", ["layer", "rms"])
def test_training_lowers_the_loss(example, norm):
    losses, norms = example.train(norm, steps=12, tokens=256)
    assert losses[-1] < losses[0] - 0.5 and all(n > 0 for n in norms)


@pytest.mark.parametrize("norm", ["layer", "rms"])
def test_gradients_against_64_bits(example, norm):
    """The 16-bit steps are taken where the library takes them (E and its
    gradient); dE is within 5e-3 of 64 bits there (Frobenius norm) and rounded
    to bf16, off by 2^-8 more at most, which the norm's linear backward keeps
    relative to its input up to its condition; 2e-2 bounds both for these
    well-scaled rows."""
    torch.manual_seed(3)
    D, V = 128, 1000
    head = example.Head(D, V, norm)
    hidden = torch.randn(3, 41, D, device="cuda", requires_grad=True)
    targets = torch.randint(0, V, (3, 41), device="cuda")
    targets[:, ::9] = -100
    with torch.no_grad():
        head.weight.add_(0.2 * torch.randn(D, device="cuda"))
    loss = head(hidden, targets)
    loss.backward()

    h = hidden.detach().double().requires_grad_()
    w = head.weight.detach().double().requires_grad_()
    c = head.classifier.detach().double().requires_grad_()
    b = torch.zeros(D, dtype=torch.float64, device="cuda", requires_grad=True)
    x = h - h.mean(-1, keepdim=True) if norm == "layer" else h
    eps = 1e-5 if norm == "layer" else 1e-6
    y = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + eps) * w + b
    e = y.detach().float().bfloat16().double().requires_grad_()
    ref = torch.nn.functional.cross_entropy((e.view(-1, D) @ c.T), targets.reshape(-1), ignore_index=-100)
    ref.backward()
    y.backward(e.grad)
    assert abs(loss.item() - ref.item()) <= 1e-5 * ref.item()
    pairs = [(head.classifier.grad, c.grad, TOL_GRAD), (hidden.grad, h.grad, 2e-2), (head.weight.grad, w.grad, 2e-2)]
    if norm == "layer":
        pairs.append((head.bias.grad, b.grad, 2e-2))
    for got, want, tol in pairs:
        assert (got.double() - want).norm() <= tol * want.norm()
    # rows without a target have no gradient
    assert not hidden.grad[:, ::9].any()


def test_clipped_gradients_have_the_norm(example):
    import linear_cross_entropy_gb300 as cce
    torch.manual_seed(5)
    head = example.Head(128, 4096, "layer")
    head(torch.randn(64, 128, device="cuda"), torch.randint(0, 4096, (64,), device="cuda")).backward()
    before = cce.clip_grad_norm_(head.parameters(), 0.01)
    after = cce.cce_grad_norm([p.grad for p in head.parameters()])
    # each value is rounded to its type again: half a bf16 step relative at most
    assert before.item() > 0.01 and abs(after.item() - 0.01) <= 0.01 * (2.0 ** -8 + 1e-3)
