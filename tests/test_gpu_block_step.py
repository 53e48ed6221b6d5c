"""A training step through a layer in front of the head: transform or gated block,
norm, classifier with cross entropy, backward pass and AdamW together."""
import importlib.util
import os

import pytest
import torch

from tests import layers_util as L

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


@pytest.mark.parametrize("block", ["transform", "gated"])
@pytest.mark.parametrize("optimizer", ["sgd", "adamw", "adamw8"])
def test_training_runs(example, block, optimizer):
    losses, norms = example.train("rms", steps=3, tokens=256, block=block, optimizer=optimizer)
    assert all(v == v and v > 0 for v in losses + norms)
    assert example.train("rms", steps=3, tokens=256, block=block, optimizer=optimizer) == (losses, norms)


@pytest.mark.parametrize("block", ["transform", "gated"])
def test_gradients_against_64_bits(example, block):
    """The chain in 64 bits, rounded to 16 bits where the library does on the
    way forward.  A gradient then differs by the roundings of the way back: of dE
    (bound 5e-3 of its norm in the head's own tests), of each layer's dz and
    result (2^-8 at most of each value) and of the kept pre-activations (2^-8 of each, times
    a slope below 2 of the factor in front of it): 5e-3 and five roundings of 2^-8 =
    2.5e-2 of a gradient's norm at most, which the well-scaled linear maps between
    them keep relative up to their condition, 1.6 for random square weights' mean gain."""
    torch.manual_seed(3)
    D, V = 128, 1000
    head = example.Head(D, V, "rms")
    front = example.BLOCKS[block](D)
    hidden = torch.randn(3, 41, D, device="cuda", requires_grad=True)
    targets = torch.randint(0, V, (3, 41), device="cuda")
    targets[:, ::9] = -100
    loss = head(front(hidden), targets)
    loss.backward()

    def d(t):
        return t.detach().double().requires_grad_()

    def rounded(t):
        return t + (t.detach().float().bfloat16().double() - t.detach())

    def rms(t, w):
        return t * torch.rsqrt(t.square().mean(-1, keepdim=True) + 1e-6) * w
    h, w, c = d(hidden), d(head.weight), d(head.classifier)
    p = {k: d(v) for k, v in front.named_parameters()}
    if block == "transform":
        out = L.act64("gelu", rounded(h) @ p["weight"].T + p["bias"])
    else:
        n = rounded(rms(h, p["norm"]))
        out = rounded(L.act64("silu", n @ p["gate"].T) * (n @ p["up"].T)) @ p["down"].T + h
    e = rounded(rms(out, w))
    ref = torch.nn.functional.cross_entropy(e.view(-1, D) @ c.T, targets.reshape(-1), ignore_index=-100)
    ref.backward()
    assert abs(loss.item() - ref.item()) <= 1e-4 * ref.item()
    pairs = [(hidden.grad, h.grad), (head.weight.grad, w.grad), (head.classifier.grad, c.grad)]
    pairs += [(q.grad, p[k].grad) for k, q in front.named_parameters()]
    for got, want in pairs:
        assert (got.double() - want).norm() <= 1.6 * 2.5e-2 * want.norm()
    assert not hidden.grad[:, ::9].any()  # rows without a target have no gradient


@pytest.mark.parametrize("bits", [8, 32])
def test_captured_step(example, bits):
    """A whole step in a CUDA graph gives the eager step's parameters."""
    import linear_cross_entropy_gb300 as cce

    def make():
        torch.manual_seed(4)
        block = example.GatedBlock(64, 160)
        opt = cce.AdamW(block.parameters(), lr=1e-2, state_bits=bits, master_weights=True, capturable=True)
        return block, opt, torch.randn(70, 64, device="cuda")

    def step(block, opt, x):
        g = torch.autograd.grad(block(x).square().mean(), list(block.parameters()))
        for q, gq in zip(block.parameters(), g):
            q.grad = gq
        opt.step(grad_norm=cce.cce_grad_norm(g), max_norm=0.5)

    a, opt_a, x = make()
    for _ in range(4):
        step(a, opt_a, x)
    b, opt_b, x = make()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(b, opt_b, x)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step(b, opt_b, x)
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    for q, r in zip(a.parameters(), b.parameters()):
        assert torch.equal(q, r)
