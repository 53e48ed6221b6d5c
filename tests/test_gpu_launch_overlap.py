"""Chains of calls in which each reads what the call before it writes, behind a
long call, so that the launches overlap.  The buffers are fixed, hold NaN before
each chain, and the inputs alternate: whoever reads too early reads NaN or the
other input's values.  What is compared with are the same calls with a wait for
the GPU after each, bit by bit."""
import pytest
import torch

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16
EPS = 1e-5


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    from tests.conftest import build_library
    build_library()
    from linear_cross_entropy_gb300 import _lib
    return _lib.load()


def _randn(seed, *shape):
    return torch.randn(shape, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda").to(BF16)


def _nan(*shape, dtype=BF16):
    return torch.full(shape, float("nan"), device="cuda", dtype=dtype)


def _stream():
    return torch.cuda.current_stream().cuda_stream


class Norm:
    """Layer norm through the C ABI into given buffers."""

    def __init__(self, lib, N, D):
        self.lib, self.N, self.D = lib, N, D
        self.need = lib.cce_norm_backward_workspace_bytes(N, D)
        self.ws = torch.empty(self.need, device="cuda", dtype=torch.uint8)
        self.mean, self.rstd = _nan(N, dtype=torch.float32), _nan(N, dtype=torch.float32)

    def forward(self, x, w, b, y):
        assert self.lib.cce_layer_norm_forward(x.data_ptr(), self.N, self.D, 0, 2, w.data_ptr(), b.data_ptr(), 2, self.N,
                                               self.D, EPS, y.data_ptr(), 2, self.mean.data_ptr(), self.rstd.data_ptr(),
                                               _stream()) == 0

    def backward(self, dy, x, w, dx, dw, db):
        assert self.lib.cce_layer_norm_backward(dy.data_ptr(), self.N, self.D, 0, 2, x.data_ptr(), self.N, self.D, 0, 2,
                                                w.data_ptr(), 2, self.mean.data_ptr(), self.rstd.data_ptr(), self.N,
                                                self.D, dx.data_ptr(), dw.data_ptr(), db.data_ptr(), self.ws.data_ptr(),
                                                self.need, _stream()) == 0


class Long:
    """A call of some 90 us on buffers of its own."""

    def __init__(self, lib):
        self.norm = Norm(lib, 65536, 2048)
        self.x, self.y = _randn(1, 65536, 2048), torch.empty(65536, 2048, device="cuda", dtype=BF16)
        self.w, self.b = _randn(2, 2048), _randn(3, 2048)

    def __call__(self):
        self.norm.forward(self.x, self.w, self.b, self.y)


@pytest.fixture(scope="module")
def long_call(lib):
    return Long(lib)


def _compare(chain, inputs, buffers, results, long_call, rounds=6):
    """chain(i, pause) runs the calls on inputs[i]."""
    def prepared():
        for t in buffers:
            t.fill_(float("nan"))

    want = []
    for i in range(len(inputs)):
        prepared()
        chain(inputs[i], torch.cuda.synchronize)
        torch.cuda.synchronize()
        want.append([t.clone() for t in results])
        assert all(torch.isfinite(t).all() for t in want[-1])
    assert not all(torch.equal(a, b) for a, b in zip(*want[:2]))
    got = []
    for r in range(rounds):
        prepared()
        long_call()
        chain(inputs[r % len(inputs)], lambda: None)
        got.append([t.clone() for t in results])
    torch.cuda.synchronize()
    for r in range(rounds):
        for a, b in zip(got[r], want[r % len(inputs)]):
            assert torch.equal(a, b), r


# rows of the call that reads: a block a row, persistent groups; widths: aligned, shifted, too long for registers
@pytest.mark.parametrize("rows", [1, 300, 1500])
@pytest.mark.parametrize("D", [1024, 1001, 33000])
def test_a_norm_of_a_norm(lib, long_call, rows, D):
    N = max(rows, (1 << 22) // D)
    xs = [_randn(s, N, D) for s in (10, 11)]
    w, b = _randn(12, D), _randn(13, D)
    y, z = _nan(N, D), _nan(rows, D)
    first, second = Norm(lib, N, D), Norm(lib, rows, D)

    def chain(x, pause):
        first.forward(x, w, b, y)
        pause()
        second.forward(y[N - rows:], w, b, z)

    _compare(chain, xs, [y, z], [z, second.mean, second.rstd], long_call)


@pytest.mark.parametrize("N,D", [(1, 896), (40, 1024), (3000, 1024), (3001, 1001)])
def test_gradients_read_by_the_next_norm(lib, long_call, N, D):
    """dx as the rows, dw and db as the parameters of the call behind the backward."""
    pairs = [(_randn(s, N, D), _randn(s + 1, N, D)) for s in (20, 22)]
    w, b = _randn(24, D), _randn(25, D)
    y, dx, dw, db, z = _nan(N, D), _nan(N, D), _nan(D), _nan(D), _nan(N, D)
    norm, after = Norm(lib, N, D), Norm(lib, N, D)

    def chain(pair, pause):
        norm.forward(pair[0], w, b, y)
        pause()
        norm.backward(pair[1], pair[0], w, dx, dw, db)
        pause()
        after.forward(dx, dw, db, z)

    _compare(chain, pairs, [y, dx, dw, db, z, norm.mean, norm.rstd], [dx, dw, db, z], long_call)


@pytest.mark.parametrize("N,D", [(1, 896), (33, 1001), (2000, 128)])
def test_short_calls_through_two_buffers(lib, long_call, N, D):
    """Eight short norms, each of the last one's result: more than two are resident at once."""
    xs = [_randn(s, N, D) for s in (30, 31)]
    w, b = _randn(32, D), _randn(33, D)
    p, q = _nan(N, D), _nan(N, D)
    norm = Norm(lib, N, D)

    def chain(x, pause):
        norm.forward(x, w, b, p)
        for _ in range(4):
            pause()
            norm.forward(p, w, b, q)
            pause()
            norm.forward(q, w, b, p)

    _compare(chain, xs, [p, q], [p, q, norm.rstd], long_call)


@pytest.mark.parametrize("sizes", [(1000, 77), (3_000_001, 4096, 5)])
def test_the_norm_of_gradients_just_clipped(lib, long_call, sizes):
    """The gradients are clipped in place, measured, and clipped again."""
    import linear_cross_entropy_gb300 as cce
    sources = [[_randn(s + i, n) for i, n in enumerate(sizes)] for s in (40, 50)]
    grads = [_nan(n) for n in sizes]
    results = list(grads)

    def chain(source, pause):
        for g, s in zip(grads, source):
            g.copy_(s)
        long_call()
        del results[len(grads):]
        for call in (lambda: cce.cce_clip_grads(grads, 0.5), lambda: cce.cce_grad_norm(grads),
                     lambda: cce.cce_clip_grads(grads, 0.25)):
            pause()
            results.append(call())

    _compare(chain, sources, grads, results, long_call)
