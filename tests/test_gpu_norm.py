"""Layer norm and RMS norm on the GPU against the 64-bit formulas: every type
and layout, sizes on both sides of each kernel's limits, strided rows, empty
inputs, extreme values, streams and graphs."""
import numpy as np
import pytest
import torch

from oracle import ops
from tests import ops_util as U

pytestmark = pytest.mark.gpu

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
PAIRS = [(BF16, BF16), (F16, F16), (F32, F32), (F32, BF16), (F32, F16)]


@pytest.fixture(scope="module", autouse=True)
def cce():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    from tests.conftest import build_library
    build_library()
    import linear_cross_entropy_gb300
    return linear_cross_entropy_gb300


def _randn(gen, *shape):
    return torch.randn(shape, generator=gen, device="cuda")


def _inputs(seed, shape, x_type, y_type, p_type, mean=0.2):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    D = shape[-1]
    x = (_randn(gen, *shape) * torch.exp(0.5 * _randn(gen, D)) + mean).to(x_type)
    w = (1 + 0.3 * _randn(gen, D)).to(p_type)
    b = (0.3 * _randn(gen, D)).to(p_type)
    return x, w, b, _randn(gen, *shape).to(y_type)


def _check(cce, x, w, b, dy, layer, eps=1e-5, offset=0.0, out_dtype=None):
    """Forward and direct backward against 64 bits."""
    D = x.shape[-1]
    xd = U.f64(x)
    gain = (w.double().cpu().numpy() + (0.0 if layer else offset)) if w is not None else np.ones(D)
    bias = b.double().cpu().numpy() if b is not None and layer else np.zeros(D)
    mean, rstd = ops.norm_stats(xd, eps, layer)
    if layer:
        y, m, r = cce.cce_layer_norm_forward(x, w, b, eps, out_dtype=out_dtype)
        U.within(m, mean, np.abs(xd).mean(axis=1), F32, "mean")
    else:
        y, r = cce.cce_rms_norm_forward(x, w, eps, weight_offset=offset, out_dtype=out_dtype)
    assert y.shape == x.shape and y.is_contiguous() and y.dtype == (out_dtype or x.dtype)
    U.within(y, ops.norm_forward(xd, gain, bias, mean, rstd), U.forward_magnitude(xd, gain, bias, mean, rstd), y.dtype,
             "y")
    if dy is None:
        return
    # the backward on the statistics that the forward gave, taken as they are
    rd = r.double().cpu().numpy()
    md = m.double().cpu().numpy() if layer else np.zeros(rd.shape)
    if layer:
        dx, dw, db = cce.cce_layer_norm_backward(dy, x, w, m, r, param_dtype=None if w is not None else F32)
    else:
        dx, dw = cce.cce_rms_norm_backward(dy, x, w, r, weight_offset=offset)
        assert (dw is None) == (w is None)
    gd = U.f64(dy)
    ex, ew, eb = ops.norm_backward(gd, xd, gain, md, rd, layer)
    mx, mw, mb = U.backward_magnitudes(gd, xd, gain, md, rd, layer)
    assert dx.shape == x.shape and dx.dtype == x.dtype
    U.within(dx, ex, mx, dx.dtype, "dx")
    if dw is not None:
        U.within(dw, ew, mw, dw.dtype, "dw")
    if layer:
        U.within(db, eb, mb, db.dtype, "db")


@pytest.mark.parametrize("layer", [True, False])
@pytest.mark.parametrize("N,D", [(1, 1), (1, 8), (3, 5), (1, 896), (2, 64), (33, 63), (5, 128), (1000, 128), (17, 256),
                                 (700, 1001), (33, 1024), (257, 2304), (1, 4096), (40, 4096), (9, 4097), (19, 6152),
                                 (3, 8200), (5, 8191), (4, 16384), (5, 16392), (3, 20001), (2, 33000), (1, 70000)])
def test_sizes(cce, layer, N, D):
    x, w, b, dy = _inputs(N * 7919 + D, (N, D), BF16, BF16, BF16)
    _check(cce, x, w, b, dy, layer)


@pytest.mark.parametrize("layer", [True, False])
@pytest.mark.parametrize("x_type,y_type", PAIRS)
@pytest.mark.parametrize("p_type", [BF16, F16, F32])
@pytest.mark.parametrize("D", [40, 333, 1000, 2052, 5000, 9000, 17000])
def test_types(cce, layer, x_type, y_type, p_type, D):
    x, w, b, dy = _inputs(D, (21, D), x_type, y_type, p_type)
    _check(cce, x, w, b, dy, layer, out_dtype=y_type)


@pytest.mark.parametrize("N,D", [(5000, 64), (3001, 896), (20000, 130), (4099, 2304)])
def test_many_rows(cce, N, D):
    for layer in (True, False):
        x, w, b, dy = _inputs(N, (N, D), BF16, BF16, F32)
        _check(cce, x, w, b, dy, layer)


@pytest.mark.parametrize("layer", [True, False])
@pytest.mark.parametrize("x_type,y_type", PAIRS)
@pytest.mark.parametrize("N,D", [(5001, 333), (2003, 1003), (1700, 65), (333, 4099), (190, 9001)])
def test_many_odd_rows(cce, layer, x_type, y_type, N, D):
    """Rows that start at any place of a 16-byte word, several to a thread group."""
    x, w, b, dy = _inputs(N + D, (N, D), x_type, y_type, F32)
    _check(cce, x, w, b, dy, layer, out_dtype=y_type)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_odd_rows_at_a_pitch(cce, dtype):
    """Odd widths inside wider matrices: at pitches that keep every matrix's rows
    alike (a multiple of 16 bytes more), at others, and overlapping windows."""
    for D, pitch in [(333, 333 + 16), (333, 340), (1001, 1001 + 8), (129, 250)]:
        x, w, b, dy = _inputs(D + pitch, (700, pitch), dtype, dtype, dtype)
        for layer in (True, False):
            _check(cce, x[:, :D], w[:D].contiguous(), b[:D].contiguous(), dy[:, :D].contiguous(), layer)
            _check(cce, x[:, :D], w[:D].contiguous(), b[:D].contiguous(), dy[:, :D], layer)
    flat, w, b, dy = _inputs(3, (2000,), dtype, dtype, dtype)
    windows = flat.as_strided((900, 129), (1, 1))
    _check(cce, windows, w[:129].contiguous(), b[:129].contiguous(), torch.randn(900, 129, device="cuda").to(dtype), True)


def _among_nans(t, run, before, pitch, gap):
    """The rows of t at `pitch`, every `run` of them `gap` apart, `before` elements
    into a buffer of NaNs that ends with the last row."""
    N, D = t.shape
    runs, outer = N // run, run * pitch + gap
    buf = torch.full((before + runs * outer - gap - pitch + D,), float("nan"), device="cuda", dtype=t.dtype)
    view = buf.as_strided((runs, run, D), (outer, pitch, 1), before)
    view.copy_(t.view(runs, run, D))
    return view


@pytest.mark.parametrize("layer", [True, False])
@pytest.mark.parametrize("x_type,y_type", PAIRS)
@pytest.mark.parametrize("N,D", [(1400, 64), (2100, 65), (1400, 333), (1400, 1001), (840, 1000), (700, 2049), (700, 5003),
                                 (350, 13001)])
def test_matrices_shifted_apart(cce, layer, x_type, y_type, N, D):
    """Rows of x and dy at starts that no vector divides, each matrix's in its own
    way, in runs, among NaNs; sizes past those of the kernels for few rows."""
    x, w, b, dy = _inputs(N + D, (N, D), x_type, y_type, BF16)
    for run, x_place, dy_place in [(N, (1, D, 0), (0, D, 0)), (7, (0, D, D), (0, D, D)),
                                   (70, (5, D + 3, 1), (2, D, 6)), (14, (0, D, 0), (7, D + 1, 5))]:
        _check(cce, _among_nans(x, run, *x_place), w, b, _among_nans(dy, run, *dy_place), layer)


@pytest.mark.parametrize("layer", [True, False])
@pytest.mark.parametrize("y_at,dx_at", [(64, 65), (67, 64), (61, 70)])
@pytest.mark.parametrize("N,D", [(700, 1001), (1500, 136), (2000, 67)])
def test_results_off_their_alignment(cce, layer, y_at, dx_at, N, D):
    """y and dx at any element of a buffer, through the C ABI."""
    from linear_cross_entropy_gb300 import _lib
    lib = _lib.load()
    x, w, b, dy = _inputs(N + D, (N, D), BF16, BF16, BF16)
    y, dx = (torch.full((at + N * D + 64,), 7.0, device="cuda", dtype=BF16) for at in (y_at, dx_at))
    dw, db = (torch.empty(D, device="cuda", dtype=BF16) for _ in range(2))
    mean, rstd = (torch.empty(N, device="cuda") for _ in range(2))
    need = lib.cce_norm_backward_workspace_bytes(N, D)
    ws = torch.empty(need, device="cuda", dtype=torch.uint8)
    stream = torch.cuda.current_stream().cuda_stream
    rows, y_p, dx_p = (N, D, 0), y.data_ptr() + 2 * y_at, dx.data_ptr() + 2 * dx_at
    if layer:
        assert lib.cce_layer_norm_forward(x.data_ptr(), *rows, 2, w.data_ptr(), b.data_ptr(), 2, N, D, 1e-5, y_p, 2,
                                          mean.data_ptr(), rstd.data_ptr(), stream) == 0
        assert lib.cce_layer_norm_backward(dy.data_ptr(), *rows, 2, x.data_ptr(), *rows, 2, w.data_ptr(), 2,
                                           mean.data_ptr(), rstd.data_ptr(), N, D, dx_p, dw.data_ptr(), db.data_ptr(),
                                           ws.data_ptr(), need, stream) == 0
    else:
        assert lib.cce_rms_norm_forward(x.data_ptr(), *rows, 2, w.data_ptr(), 2, 0.0, N, D, 1e-5, y_p, 2,
                                        rstd.data_ptr(), stream) == 0
        assert lib.cce_rms_norm_backward(dy.data_ptr(), *rows, 2, x.data_ptr(), *rows, 2, w.data_ptr(), 2, 0.0,
                                         rstd.data_ptr(), N, D, dx_p, dw.data_ptr(), ws.data_ptr(), need, stream) == 0
    xd, gd, gain = U.f64(x), U.f64(dy), w.double().cpu().numpy()
    bias = b.double().cpu().numpy() if layer else np.zeros(D)
    m, r = ops.norm_stats(xd, 1e-5, layer)
    U.within(y[y_at:-64].view(N, D), ops.norm_forward(xd, gain, bias, m, r), U.forward_magnitude(xd, gain, bias, m, r),
             BF16, "y")
    rd = rstd.double().cpu().numpy()
    md = mean.double().cpu().numpy() if layer else np.zeros(N)
    for got, exact, size, name in zip((dx[dx_at:-64].view(N, D), dw, db), ops.norm_backward(gd, xd, gain, md, rd, layer),
                                      U.backward_magnitudes(gd, xd, gain, md, rd, layer), ("dx", "dw", "db")):
        if layer or name != "db":
            U.within(got, exact, size, BF16, name)
    for t, at in ((y, y_at), (dx, dx_at)):
        assert (t[:at] == 7.0).all() and (t[-64:] == 7.0).all()


@pytest.mark.parametrize("N,D", [(1, 65), (3, 333), (500, 1001), (2000, 67), (40, 4097)])
def test_nothing_is_written_outside_the_results(cce, N, D):
    """y, dx and the parameters' gradients between guard values, through the C ABI."""
    from linear_cross_entropy_gb300 import _lib
    lib = _lib.load()
    x, w, b, dy = _inputs(N + D, (N, D), BF16, BF16, BF16)
    guard = 64
    y, dx = (torch.full((guard + N * D + guard,), 7.0, device="cuda", dtype=BF16) for _ in range(2))
    dw, db = (torch.full((guard + D + guard,), 7.0, device="cuda", dtype=BF16) for _ in range(2))
    mean, rstd = (torch.full((guard + N + guard,), 7.0, device="cuda") for _ in range(2))
    at = lambda t: t.data_ptr() + guard * t.element_size()  # noqa: E731
    stream = torch.cuda.current_stream().cuda_stream
    assert lib.cce_layer_norm_forward(x.data_ptr(), N, D, 0, 2, w.data_ptr(), b.data_ptr(), 2, N, D, 1e-5, at(y), 2,
                                      at(mean), at(rstd), stream) == 0
    need = lib.cce_norm_backward_workspace_bytes(N, D)
    ws = torch.full((need + 4096,), 85, device="cuda", dtype=torch.uint8)
    assert lib.cce_layer_norm_backward(dy.data_ptr(), N, D, 0, 2, x.data_ptr(), N, D, 0, 2, w.data_ptr(), 2, at(mean),
                                       at(rstd), N, D, at(dx), at(dw), at(db), ws.data_ptr(), need, stream) == 0
    want = cce.cce_layer_norm_forward(x, w, b)
    dwant = cce.cce_layer_norm_backward(dy, x, w, *want[1:])
    for t, ref in zip((y, mean, rstd, dx, dw, db), want + dwant):
        assert (t[:guard] == 7.0).all() and (t[-guard:] == 7.0).all()
        assert torch.equal(t[guard:-guard], ref.reshape(-1))
    assert (ws[need:] == 85).all()


def test_weight_offset_and_missing_parameters(cce):
    x, w, b, dy = _inputs(5, (37, 520), BF16, BF16, BF16)
    _check(cce, x, w - 1, None, dy, False, offset=1.0)
    _check(cce, x, None, None, dy, True)
    _check(cce, x, None, b, dy, True)
    _check(cce, x, w, None, dy, True)
    _check(cce, x, None, None, dy, False, offset=1.0)


@pytest.mark.parametrize("layer", [True, False])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_strided_rows(cce, layer, dtype):
    """Rows of views: shifted sequences, column slices on and off 16-byte
    boundaries, every other row, transposed leading dimensions, expanded rows."""
    x, w, b, dy = _inputs(11, (4, 9, 640), dtype, dtype, dtype)
    cuts = [lambda t: t[:, :-1], lambda t: t[:, 1:], lambda t: t[..., :320], lambda t: t[..., 8:328],
            lambda t: t[..., 3:323], lambda t: t[:, ::2, 1:301], lambda t: t.transpose(0, 1), lambda t: t[0, 0],
            lambda t: t[..., ::2], lambda t: t[1:2, :5].expand(3, 5, 640)]
    for cut in cuts:
        xv, gv = cut(x), cut(dy)
        D = xv.shape[-1]
        _check(cce, xv, w[:D].contiguous(), b[:D].contiguous(), gv, layer)
        _check(cce, xv, w[:D].contiguous(), b[:D].contiguous(), gv.contiguous(), layer)


def test_parameters_off_their_alignment(cce):
    x, w, b, dy = _inputs(12, (19, 65), BF16, BF16, BF16)
    _check(cce, x[:, 1:].contiguous(), w[1:], b[1:], dy[:, 1:].contiguous(), True)
    _check(cce, x[:, 1:].contiguous(), w[1:], None, dy[:, 1:].contiguous(), False)


def test_no_rows(cce):
    w = torch.ones(48, device="cuda", dtype=BF16)
    x = torch.empty(0, 48, device="cuda", dtype=BF16)
    y, m, r = cce.cce_layer_norm_forward(x, w, w)
    assert y.shape == (0, 48) and m.numel() == 0
    dx, dw, db = cce.cce_layer_norm_backward(x, x, w, m, r)
    assert dx.shape == (0, 48) and not dw.any() and not db.any()
    y, r = cce.cce_rms_norm_forward(x.view(3, 0, 48), w)
    assert y.shape == (3, 0, 48)
    dx, dw = cce.cce_rms_norm_backward(x, x, w, r)
    assert not dw.any()


def test_only_what_is_needed(cce):
    x, w, b, dy = _inputs(13, (50, 264), BF16, BF16, F32)
    y, m, r = cce.cce_layer_norm_forward(x, w, b)
    full = cce.cce_layer_norm_backward(dy, x, w, m, r)
    for need in [(True, False, False), (False, True, False), (False, False, True), (True, True, False),
                 (False, True, True)]:
        part = cce.cce_layer_norm_backward(dy, x, w, m, r, need_dx=need[0], need_dweight=need[1], need_dbias=need[2])
        for want, p, f in zip(need, part, full):
            assert torch.equal(p, f) if want else p is None
    y2, m2, r2 = cce.cce_layer_norm_forward(x, w, b, stats=False)
    assert torch.equal(y, y2) and m2 is None and r2 is None


def test_mean_far_from_zero_does_not_cancel(cce):
    """Rows around 1000 with deviations around 1: sums of squares would leave
    nothing of the variance in fp32; the squared deviations keep it."""
    for D in (100, 896, 4096, 30000):
        x, w, b, dy = _inputs(D, (6, D), F32, F32, F32, mean=1000.0)
        _check(cce, x, w, b, dy, True)


def test_constant_and_zero_rows(cce):
    x = torch.zeros(4, 136, device="cuda", dtype=F32)
    x[1] = 7.0
    x[2] = -2.5
    w = torch.full((136,), 2.0, device="cuda")
    b = torch.full((136,), 0.5, device="cuda")
    y, m, r = cce.cce_layer_norm_forward(x, w, b, 1e-5)
    assert torch.equal(y, torch.full_like(y, 0.5)) and m.tolist() == [0.0, 7.0, -2.5, 0.0]
    dx, dw, db = cce.cce_layer_norm_backward(torch.ones_like(x), x, w, m, r)
    assert torch.isfinite(dx).all() and not dw.any() and torch.equal(db, torch.full_like(db, 4.0))
    y, r = cce.cce_rms_norm_forward(x[:1], w, 1e-6)
    assert not y.any()


def test_a_bad_row_stays_its_own(cce):
    """NaN and infinities spoil their row and the parameters' gradients, no other row."""
    x, w, b, dy = _inputs(17, (40, 200), BF16, BF16, BF16)
    good = cce.cce_layer_norm_forward(x, w, b)
    gdx = cce.cce_layer_norm_backward(dy, x, w, *good[1:])[0]
    x2 = x.clone()
    x2[3, 5], x2[9, 0], x2[39, 199] = float("nan"), float("inf"), float("-inf")
    y, m, r = cce.cce_layer_norm_forward(x2, w, b)
    dx, dw, _ = cce.cce_layer_norm_backward(dy, x2, w, m, r)
    for n in range(40):
        if n in (3, 9, 39):
            assert torch.isnan(y[n]).any() and torch.isnan(dx[n]).any()
        else:
            assert torch.equal(y[n], good[0][n]) and torch.equal(dx[n], gdx[n])
    assert torch.isnan(dw).all()


@pytest.mark.parametrize("layer", [True, False])
def test_autograd_matches_the_direct_calls(cce, layer):
    x, w, b, dy = _inputs(19, (3, 11, 328), BF16, BF16, F32)
    leaves = [t.clone().requires_grad_() for t in ((x, w, b) if layer else (x, w))]
    y = cce.layer_norm(*leaves) if layer else cce.rms_norm(*leaves, weight_offset=0.5)
    y.backward(dy)
    if layer:
        y0, m, r = cce.cce_layer_norm_forward(x, w, b)
        want = cce.cce_layer_norm_backward(dy, x, w, m, r)
    else:
        y0, r = cce.cce_rms_norm_forward(x, w, weight_offset=0.5)
        want = cce.cce_rms_norm_backward(dy, x, w, r, weight_offset=0.5)
    assert torch.equal(y, y0)
    for leaf, g in zip(leaves, want):
        assert torch.equal(leaf.grad, g) and leaf.grad.dtype == leaf.dtype
    # an expanded upstream gradient, some leaves frozen
    leaves = [t.clone() for t in ((x, w, b) if layer else (x, w))]
    leaves[1].requires_grad_()
    y = cce.layer_norm(*leaves) if layer else cce.rms_norm(*leaves)
    y.float().sum().backward()
    assert leaves[0].grad is None and leaves[1].grad is not None
    with torch.no_grad():
        assert not (cce.layer_norm(*leaves) if layer else cce.rms_norm(*leaves)).requires_grad
    # a bias that trains alone
    if layer:
        b2 = b.clone().requires_grad_()
        cce.layer_norm(x, None, b2).backward(dy)
        U.within(b2.grad, U.f64(dy).sum(axis=0), np.abs(U.f64(dy)).sum(axis=0), F32, "db")


def test_autograd_without_parameters(cce):
    """Every choice of parameters and of leaves that train."""
    x, w, b, dy = _inputs(21, (9, 96), F32, F32, F32)
    for have_w, have_b in [(False, False), (True, False), (False, True), (True, True)]:
        for train in [(True, True, True), (True, False, False), (False, True, True), (False, True, False),
                      (False, False, True)]:
            leaves = [t.clone().requires_grad_(r) for t, r in zip((x, w, b), train)]
            args = [leaves[0], leaves[1] if have_w else None, leaves[2] if have_b else None]
            if not any(a is not None and a.requires_grad for a in args):
                continue
            cce.layer_norm(*args).backward(dy)
            y, m, r = cce.cce_layer_norm_forward(x, w if have_w else None, b if have_b else None)
            want = cce.cce_layer_norm_backward(dy, x, w if have_w else None, m, r, param_dtype=None if have_w else F32)
            for leaf, a, g in zip(leaves, args, want):
                assert (leaf.grad is None) == (a is None or not a.requires_grad)
                if leaf.grad is not None:
                    assert torch.equal(leaf.grad, g)
    x2 = x.clone().requires_grad_()
    cce.rms_norm(x2).backward(dy)
    y, r = cce.cce_rms_norm_forward(x)
    assert torch.equal(x2.grad, cce.cce_rms_norm_backward(dy, x, None, r)[0])


def test_step_captured_into_a_graph(cce):
    """Forward and backward of the autograd form in a graph, while an eager graph
    of other leaves is alive.  (One of the same leaves may not be: their
    accumulation nodes would bring its stream into the capture.)"""
    x, w, b, dy = _inputs(45, (64, 333), BF16, BF16, F32)
    others = [t.clone().requires_grad_() for t in (x, w, b)]
    alive = cce.layer_norm(*others)
    leaves = [t.clone().requires_grad_() for t in (x, w, b)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        torch.autograd.grad(cce.layer_norm(*leaves), leaves, dy)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = torch.autograd.grad(cce.layer_norm(*leaves), leaves, dy)
    graph.replay()
    want = torch.autograd.grad(alive, others, dy)
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_no_second_derivative(cce):
    x, w, b, dy = _inputs(23, (4, 64), F32, F32, F32)
    x.requires_grad_()
    (g,) = torch.autograd.grad(cce.layer_norm(x, w, b), x, dy, create_graph=True)
    with pytest.raises(RuntimeError):
        g.sum().backward()


@pytest.mark.parametrize("layer", [True, False])
def test_gradient_against_differences_of_the_kernel(cce, layer):
    """The derivative along a direction from two forward calls.  The two-sided
    difference of step h is off by its truncation, which the 64-bit formula
    gives, and by the roundings of y over 2h."""
    N, D, h, eps = 6, 200, 2.0 ** -5, 1e-5
    x, w, b, dy = _inputs(29, (N, D), F32, F32, F32)
    v = torch.randn(N, D, generator=torch.Generator(device="cuda").manual_seed(1), device="cuda")
    lo, hi = x - h * v, x + h * v  # as rounded; the true direction is (hi - lo) / 2h
    c = U.f64(dy)

    def f(t):
        y = cce.layer_norm(t, w, b, eps) if layer else cce.rms_norm(t, w, eps)
        return float((U.f64(y) * c).sum())

    gain = w.double().cpu().numpy()
    bias = b.double().cpu().numpy() if layer else np.zeros(D)

    def exact(t):
        t = U.f64(t)
        return float((ops.norm_forward(t, gain, bias, *ops.norm_stats(t, eps, layer)) * c).sum())

    xd = U.f64(x)
    mean, rstd = ops.norm_stats(xd, eps, layer)
    ex, _, _ = ops.norm_backward(c, xd, gain, mean, rstd, layer)
    direction = (U.f64(hi) - U.f64(lo)) / (2 * h)
    truncation = abs((exact(hi) - exact(lo)) / (2 * h) - float((ex * direction).sum()))
    rounding = sum(float((np.abs(c) * U.U32 * U.forward_magnitude(U.f64(t), gain, bias,
                                                                  *ops.norm_stats(U.f64(t), eps, layer))).sum())
                   for t in (lo, hi)) / (2 * h)
    x.requires_grad_()
    y = cce.layer_norm(x, w, b, eps) if layer else cce.rms_norm(x, w, eps)
    (dx,) = torch.autograd.grad(y, x, dy)
    slope = float((U.f64(dx) * direction).sum())
    own = float((U.U32 * U.backward_magnitudes(c, xd, gain, mean, rstd, layer)[0] * np.abs(direction)).sum())
    assert abs((f(hi) - f(lo)) / (2 * h) - slope) <= truncation + rounding + own


def test_repeated_calls_are_bitwise_equal(cce):
    x, w, b, dy = _inputs(31, (3000, 896), BF16, BF16, F32)
    first = None
    for _ in range(3):
        y, m, r = cce.cce_layer_norm_forward(x, w, b)
        got = (y, m, r) + cce.cce_layer_norm_backward(dy, x, w, m, r)
        first = first or got
        assert all(torch.equal(a, b) for a, b in zip(got, first))


def test_on_another_stream(cce):
    x, w, b, dy = _inputs(37, (513, 1024), BF16, BF16, BF16)
    want = cce.cce_layer_norm_forward(x, w, b)
    dwant = cce.cce_layer_norm_backward(dy, x, w, *want[1:])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = cce.cce_layer_norm_forward(x, w, b)
        dgot = cce.cce_layer_norm_backward(dy, x, w, *got[1:])
    got2 = cce.cce_rms_norm_forward(x, w, stream=s)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want + dwant, got + dgot))
    assert torch.equal(got2[0], cce.cce_rms_norm_forward(x, w)[0])


@pytest.mark.parametrize("rows", [1, 300, 5000])
@pytest.mark.parametrize("D", [1024, 1001, 20000])
def test_calls_that_read_what_the_call_before_writes(cce, rows, D):
    """Long calls, each with a short one behind it that reads the rows written last."""
    N = (1 << 25) // D
    x, w, b, dy = _inputs(81, (N, D), BF16, BF16, BF16)
    y, mean, rstd = cce.cce_layer_norm_forward(x, w, b)
    dx, dw, db = cce.cce_layer_norm_backward(dy, x, w, mean, rstd)
    torch.cuda.synchronize()
    last = [cce.cce_layer_norm_forward(t[-rows:], w, b, 1e-5)[0] for t in (y, dx)]
    norm = cce.cce_grad_norm([dx, dw, db])
    torch.cuda.synchronize()
    for _ in range(3):
        del y, dx
        y, mean, rstd = cce.cce_layer_norm_forward(x, w, b)
        after_y = cce.cce_layer_norm_forward(y[-rows:], w, b, 1e-5)[0]
        dx, dw, db = cce.cce_layer_norm_backward(dy, x, w, mean, rstd)
        after_dx = cce.cce_layer_norm_forward(dx[-rows:], w, b, 1e-5)[0]
        dx.fill_(float("nan"))  # what a late reader would see
        dx, dw, db = cce.cce_layer_norm_backward(dy, x, w, mean, rstd)
        after_norm = cce.cce_grad_norm([dx, dw, db])
        assert torch.equal(after_y, last[0]) and torch.equal(after_dx, last[1])
        assert torch.equal(after_norm, norm)


def test_captured_into_a_graph(cce):
    """Forward and backward in one graph, replayed on new values, while an
    eager graph of other leaves is alive."""
    x, w, b, dy = _inputs(41, (300, 2304), BF16, BF16, BF16)
    alive = cce.layer_norm(x.clone().requires_grad_(), w, b)
    cce.cce_layer_norm_backward(dy, x, w, *cce.cce_layer_norm_forward(x, w, b)[1:])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, m, r = cce.cce_layer_norm_forward(x, w, b)
        dx, dw, db = cce.cce_layer_norm_backward(dy, x, w, m, r)
    x.copy_(_inputs(42, (300, 2304), BF16, BF16, BF16)[0])
    graph.replay()
    want = cce.cce_layer_norm_forward(x, w, b)
    dwant = cce.cce_layer_norm_backward(dy, x, w, *want[1:])
    assert all(torch.equal(a, b) for a, b in zip((y, m, r, dx, dw, db), want + dwant))
    assert alive.requires_grad


def test_rows_past_two_to_the_31_elements(cce):
    """Offsets need 64 bits: the last rows of a 2.3-billion-element input."""
    N, D = 70001, 32768
    x = torch.empty(N, D, device="cuda", dtype=BF16)
    for i in range(0, N, 10000):
        x[i:i + 10000].normal_()
    w = torch.full((D,), 1.5, device="cuda", dtype=BF16)
    y, r = cce.cce_rms_norm_forward(x, w)
    dx, _ = cce.cce_rms_norm_backward(y, x, w, r, need_dweight=False)
    for rows in (slice(0, 3), slice(65535, 65538), slice(N - 3, N)):
        ys, rs = cce.cce_rms_norm_forward(x[rows].clone(), w)
        assert torch.equal(y[rows], ys) and torch.equal(r[rows], rs)
        assert torch.equal(dx[rows], cce.cce_rms_norm_backward(ys, x[rows].clone(), w, rs, need_dweight=False)[0])


def test_refusals_on_the_gpu(cce):
    x, w, b, dy = _inputs(43, (4, 64), BF16, BF16, BF16)
    y, m, r = cce.cce_layer_norm_forward(x, w, b)
    bad = [lambda: cce.layer_norm(x.double(), w), lambda: cce.layer_norm(x, w[:32]), lambda: cce.layer_norm(x, w.cpu()),
           lambda: cce.layer_norm(x, w, b.float()), lambda: cce.layer_norm(x, w.double()),
           lambda: cce.layer_norm(x, w, out_dtype=F32), lambda: cce.layer_norm(x, w, out_dtype=F16),
           lambda: cce.rms_norm(x.long(), w), lambda: cce.rms_norm(x, w.view(1, 64)),
           lambda: cce.rms_norm(x, w.expand(2, 64)[:, 0]), lambda: cce.rms_norm(x[:, :0]),
           lambda: cce.rms_norm(torch.zeros((), device="cuda")),
           lambda: cce.cce_layer_norm_backward(dy.float(), x, w, m, r),
           lambda: cce.cce_layer_norm_backward(dy[:2], x, w, m, r),
           lambda: cce.cce_layer_norm_backward(dy, x, w, m[:2], r),
           lambda: cce.cce_layer_norm_backward(dy, x, w, m, r.half()),
           lambda: cce.cce_rms_norm_backward(dy.cpu(), x, w, r)]
    for call in bad:
        with pytest.raises(ValueError):
            call()
    with pytest.raises(cce.CCEError):
        cce.layer_norm(x, w, b, eps=-1.0)
    with pytest.raises(cce.CCEError):
        cce.rms_norm(x, w, weight_offset=float("nan"))
