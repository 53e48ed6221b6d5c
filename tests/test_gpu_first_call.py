"""The first call of a process, in a captured graph."""
import os
import subprocess
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CODE = """
import torch, linear_cross_entropy_gb300 as cce
x, w = (torch.randn(n, 128, device="cuda").bfloat16() for n in (300, 512))
t = torch.randint(0, 512, (300,), device="cuda")
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    first = {first}
graph.replay()
torch.cuda.synchronize()
captured = first.clone()
assert torch.equal(captured, {first})
loss = cce.linear_cross_entropy(x, w, t)
assert torch.isfinite(loss)
cce.raise_pending_errors()
"""


@pytest.mark.parametrize("call", ['cce.linear(x, w, activation="gelu")', "cce.gated_linear(x, w, w)"])
def test_captured(call):
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    from tests.conftest import build_library
    build_library()
    done = subprocess.run([sys.executable, "-c", CODE.format(first=call)], cwd=ROOT, capture_output=True, text=True, timeout=120)
    assert done.returncode == 0, done.stderr[-2000:]
