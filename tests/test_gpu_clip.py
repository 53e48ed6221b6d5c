"""The global gradient norm and clipping on the GPU against 64 bits.

Bounds, fixed before any run: a thread adds at most 66 squares in fp32 before
it goes on in fp64, so the sum of squares is off by at most 66 * 2^-24 and the
norm by half of that plus its rounding, below 2^-18; the factor by that and two
roundings, below 2^-17; a clipped value by that and its rounding to its type
(finfo.eps / 2 relative, half a subnormal step at least)."""
import math

import numpy as np
import pytest
import torch

from oracle import ops

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


def _grads(seed, shapes, dtypes, scale=1.0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return [(scale * torch.randn(s, generator=gen, device="cuda")).to(dtypes[i % len(dtypes)])
            for i, s in enumerate(shapes)]


def _check_norm(norm, grads, norm_type=2.0):
    want = ops.global_norm([_d(g) for g in grads], norm_type)
    assert norm.shape == () and norm.dtype == F32
    assert abs(norm.item() - want) <= 2.0 ** -18 * want, (norm.item(), want)
    return want


def _check_clipped(outs, before, norm, max_norm, eps=1e-6):
    f = ops.clip_factor(norm, max_norm, eps)
    for o, b in zip(outs, before):
        fi = torch.finfo(o.dtype)
        want = b * f
        tol = np.abs(want) * (fi.eps / 2 + 2.0 ** -16) + fi.smallest_normal * fi.eps / 2
        assert (np.abs(_d(o) - want) <= tol).all()


SHAPES = {
    "one value": [(1,)],
    "small": [(7,), (128,), (3, 5, 7)],
    "chunk edges": [(4095,), (4096,), (4097,), (16383,), (16384,), (16385,), (2, 16384)],
    "head": [(4096, 128), (128,), (128,)],
    "large": [(1000, 5003), (4097, 896), (1,), (65537,), (12, 16384)],
    "33 tensors": [(i * 37 + 1,) for i in range(33)],
    "1200 tensors": [(i % 301 + 1, 3) for i in range(1200)],
    "empty among others": [(0,), (5, 0, 3), (17,), (0, 4), (300, 3)],
}


@pytest.mark.parametrize("dtypes", [(BF16,), (F16,), (F32,), (BF16, F32, F16)])
@pytest.mark.parametrize("shapes", list(SHAPES))
@pytest.mark.parametrize("norm_type", [2.0, math.inf])
def test_norm_and_clipping(cce, shapes, dtypes, norm_type):
    grads = _grads(len(shapes), SHAPES[shapes], dtypes)
    want = _check_norm(cce.cce_grad_norm(grads, norm_type), grads, norm_type)
    before = [_d(g) for g in grads]
    # into other tensors of another type, with the gradients left alone
    outs = [torch.full(g.shape, 7.0, device="cuda", dtype=BF16 if g.dtype == F32 else F32) for g in grads]
    norm = cce.cce_clip_grads(grads, 0.3 * want, norm_type, out=outs)
    _check_norm(norm, grads, norm_type)
    _check_clipped(outs, before, want, 0.3 * want)
    assert all((_d(g) == b).all() for g, b in zip(grads, before))
    # in place
    _check_norm_value = cce.cce_clip_grads(grads, 0.3 * want, norm_type)
    assert torch.equal(_check_norm_value, norm)
    _check_clipped(grads, before, want, 0.3 * want)


@pytest.mark.parametrize("out_dtype", [BF16, F16, F32])
@pytest.mark.parametrize("in_dtype", [BF16, F16, F32])
def test_off_alignment(cce, in_dtype, out_dtype):
    """Views of flat buffers that start at any element, as buckets of odd sizes give them."""
    flat = _grads(3, [(60011,)], (in_dtype,))[0]
    oflat = torch.empty(60011, device="cuda", dtype=out_dtype)
    sizes = [1, 3, 5000, 17, 16384 + 9, 8, 20001, 2, 10000]
    starts = np.cumsum([0] + sizes[:-1]) + np.arange(len(sizes))  # one element left between
    grads = [flat[a:a + n] for a, n in zip(starts, sizes)]
    outs = [oflat[a:a + n] for a, n in zip(starts, sizes)]
    oflat.fill_(9.0)
    want = _check_norm(cce.cce_clip_grads(grads, 5.0, out=outs), grads)
    _check_clipped(outs, [_d(g) for g in grads], want, 5.0)
    for a in starts[1:]:
        assert oflat[a - 1].item() == 9.0
    before = [_d(g) for g in grads]
    rest = flat[starts[1:] - 1].clone()
    cce.cce_clip_grads(grads, 5.0)
    _check_clipped(grads, before, want, 5.0)
    assert torch.equal(flat[starts[1:] - 1], rest)


def test_strided_gradients(cce):
    base = _grads(5, [(6, 33, 40)], (BF16,))[0]
    cuts = [lambda t: t[:, :, 3:17], lambda t: t[::2, 1:], lambda t: t.transpose(0, 2), lambda t: t[:, ::3, ::2],
            lambda t: t.permute(1, 0, 2), lambda t: t[3, 4:5, :1]]
    for cut in cuts:
        b = base.clone()
        g = cut(b)
        other = _grads(6, [(100,)], (F32,))[0]
        before = [_d(g), _d(other)]
        want = _check_norm(cce.cce_grad_norm([g, other]), [g, other])
        outs = [torch.zeros(g.shape, device="cuda", dtype=F32), torch.zeros(100, device="cuda", dtype=BF16)]
        cce.cce_clip_grads([g, other], 2.0, out=outs)
        _check_clipped(outs, before, want, 2.0)
        cce.cce_clip_grads([g, other], 2.0)
        _check_clipped([g, other], before, want, 2.0)
        kept = torch.ones_like(base, dtype=torch.bool)
        cut(kept)[...] = False
        assert torch.equal(b[kept], base[kept])
    # two interleaved column slices of one buffer, clipped in place together
    b = base.clone()
    left, right = b[..., :20], b[..., 20:]
    want = _check_norm(cce.cce_clip_grads([left, right], 1.0), [base])
    _check_clipped([b], [_d(base)], want, 1.0)
    expanded = base[0, 0].expand(50, 40)
    _check_norm(cce.cce_grad_norm([expanded]), [expanded])


def test_no_clipping_below_the_limit(cce):
    grads = _grads(7, [(5000,), (33, 77)], (BF16, F32))
    same = [g.clone() for g in grads]
    norm = cce.cce_clip_grads(grads, 1e6)
    assert norm.item() > 1 and all(torch.equal(a, b) for a, b in zip(grads, same))
    cce.cce_clip_grads(grads, math.inf)
    assert all(torch.equal(a, b) for a, b in zip(grads, same))
    outs = [torch.empty_like(g) for g in grads]
    cce.cce_clip_grads(grads, math.inf, out=outs)  # still copied
    assert all(torch.equal(a, b) for a, b in zip(outs, same))
    cce.cce_clip_grads(grads, 0.0)
    assert all(not g.any() for g in grads)
    zeros = [torch.zeros(100, device="cuda")]
    assert cce.cce_clip_grads(zeros, 1.0).item() == 0.0 and not zeros[0].any()
    assert cce.cce_grad_norm([torch.empty(0, device="cuda")]).item() == 0.0
    assert cce.cce_clip_grads([torch.empty(0, 3, device="cuda")], 1.0).item() == 0.0


def test_squares_outside_the_range_of_fp32(cce):
    """Values whose squares overflow or underflow in fp32: the norm is right."""
    for value, dtype in [(1e25, F32), (3e30, BF16), (1e-25, F32), (1e-30, BF16), (2.0 ** -140, F32), (6e-8, F16)]:
        grads = [torch.full((5000,), value, device="cuda", dtype=dtype), torch.zeros(20000, device="cuda", dtype=dtype)]
        grads[1][12345] = value
        want = ops.global_norm([_d(g) for g in grads])
        assert abs(cce.cce_grad_norm(grads).item() - want) <= 2.0 ** -18 * want + 2.0 ** -150, value
        _check_norm(cce.cce_grad_norm(grads, math.inf), grads, math.inf)
    # a few tiny values beside ordinary ones
    mixed = _grads(9, [(30000,)], (F32,))[0]
    mixed[::7] *= 1e-30
    _check_norm(cce.cce_grad_norm([mixed]), [mixed])
    big = [torch.full((64,), 3e38, device="cuda")]  # the norm itself is beyond fp32
    assert cce.cce_grad_norm(big).item() == math.inf


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("at", [0, 4999, 5000, 21383])
def test_nan_and_infinity(cce, dtype, at):
    for norm_type in (2.0, math.inf):
        for bad in (math.nan, math.inf, -math.inf):
            grads = _grads(11, [(5000,), (16384,)], (dtype,))
            (grads[0] if at < 5000 else grads[1])[at if at < 5000 else at - 5000] = bad
            norm = cce.cce_grad_norm(grads, norm_type).item()
            assert math.isnan(norm) if math.isnan(bad) else norm == math.inf
            outs = [torch.empty_like(g) for g in grads]
            cce.cce_clip_grads(grads, 1.0, norm_type, out=outs)
            if math.isnan(bad):
                assert all(torch.isnan(o).all() for o in outs)
            else:  # factor 0: the infinity gives NaN, all else 0
                assert sum(int(torch.isnan(o).sum()) for o in outs) == 1
                assert sum(int((o == 0).sum()) for o in outs) == 21383


def test_parameters_like_torch(cce):
    """clip_grad_norm_ on a module against torch's own, in fp32."""
    torch.manual_seed(0)
    nets = [torch.nn.Sequential(torch.nn.Linear(65, 130), torch.nn.LayerNorm(130), torch.nn.Linear(130, 3)).cuda()
            for _ in range(2)]
    nets[1].load_state_dict(nets[0].state_dict())
    x = torch.randn(40, 65, device="cuda")
    for n in nets:
        n(x).square().sum().backward()
        n[2].bias.grad = None
    a = cce.clip_grad_norm_(nets[0].parameters(), 0.5)
    b = torch.nn.utils.clip_grad_norm_(nets[1].parameters(), 0.5)
    torch.testing.assert_close(a, b, rtol=1e-5, atol=0)
    for p, q in zip(nets[0].parameters(), nets[1].parameters()):
        if p.grad is not None:
            torch.testing.assert_close(p.grad, q.grad, rtol=1e-5, atol=1e-9)
    nets[0][0].weight.grad[0, 0] = math.nan
    kept = nets[0][2].weight.grad.clone()
    with pytest.raises(RuntimeError, match="not clipped"):
        cce.clip_grad_norm_(nets[0].parameters(), 0.5, error_if_nonfinite=True)
    assert torch.equal(nets[0][2].weight.grad, kept)
    assert math.isnan(cce.clip_grad_norm_(nets[0].parameters(), 0.5).item())


def test_autograd_sees_the_write(cce):
    w = torch.randn(64, device="cuda", requires_grad=True)
    g = torch.randn(64, device="cuda")
    y = (w * g).sum()  # saves g
    cce.cce_clip_grads([g], 0.1)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.backward()
    with torch.inference_mode():
        h = torch.randn(64, device="cuda")
        cce.cce_clip_grads([h], 0.1)


def test_repeated_and_captured(cce):
    """Bitwise the same on every call, on another stream and from a graph, whose
    replay reads the values of then."""
    grads = _grads(13, [(4096, 128), (128,), (1001, 77)], (BF16, F32))
    first = cce.cce_grad_norm(grads)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    on_s = cce.cce_grad_norm(grads, stream=s)
    s.synchronize()
    assert torch.equal(first, cce.cce_grad_norm(grads)) and torch.equal(first, on_s)
    outs = [torch.empty_like(g, dtype=F32) for g in grads]
    cce.cce_clip_grads(grads, 1.0, out=outs)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        norm = cce.cce_clip_grads(grads, 1.0, out=outs)
    for g in grads:
        g.mul_(3.0)
    for o in outs:
        o.zero_()
    graph.replay()
    want = _check_norm(norm, grads)
    _check_clipped(outs, [_d(g) for g in grads], want, 1.0)


def test_past_two_to_the_32_bytes(cce):
    """One tensor of 2.3 billion values: chunk offsets need 64 bits."""
    n = (1 << 31) + (1 << 27) + 13
    g = torch.zeros(n, device="cuda", dtype=BF16)
    spots = [0, (1 << 30) + 1, (1 << 31) - 1, 1 << 31, n - 1]
    for i in spots:
        g[i] = 2.0
    norm = cce.cce_clip_grads([g], 1.0)
    assert abs(norm.item() - math.sqrt(20.0)) <= 2.0 ** -18 * math.sqrt(20.0)
    for i in spots:
        assert abs(g[i].item() - 2.0 / math.sqrt(20.0)) <= 2.0 ** -8
    assert int((g != 0).sum()) == len(spots)


def test_refusals_on_the_gpu(cce):
    g = torch.zeros(64, device="cuda")
    bad = [lambda: cce.cce_grad_norm([g.double()]), lambda: cce.cce_grad_norm([g, g.cpu()]),
           lambda: cce.cce_grad_norm([g.long()]), lambda: cce.cce_grad_norm([g], 1.0),
           lambda: cce.cce_grad_norm([g.to_sparse()]),
           lambda: cce.cce_clip_grads([g], 1.0, out=[g[:32]]), lambda: cce.cce_clip_grads([g], 1.0, out=[g.cpu()]),
           lambda: cce.cce_clip_grads([g[:1].expand(64)], 1.0), lambda: cce.cce_clip_grads([g], -0.5)]
    for call in bad:
        with pytest.raises(ValueError):
            call()
    for rows in ([g, g], [g[:40], g[30:]]):
        with pytest.raises(cce.CCEError):
            cce.cce_clip_grads(rows, 1.0)
    with pytest.raises(cce.CCEError):
        cce.cce_clip_grads([g[:32]], 1.0, out=[g[16:48]])
    with pytest.raises(cce.CCEError):
        cce.cce_clip_grads([g], 1.0, eps=math.nan)
