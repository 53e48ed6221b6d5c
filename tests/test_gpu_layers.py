"""Linear and gated linear layers on the GPU against 64 bits (bounds: layers_util)."""
import math

import pytest
import torch

from tests import layers_util as L

pytestmark = pytest.mark.gpu

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def cce():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    from tests.conftest import build_library
    build_library()
    import linear_cross_entropy_gb300
    yield linear_cross_entropy_gb300
    linear_cross_entropy_gb300.raise_pending_errors()


def randn(gen, *shape, scale=1.0, dtype=F32):
    return (scale * torch.randn(shape, generator=gen, device="cuda")).to(dtype)


def inputs(M, N, K, dtype, seed=0, weights=1):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    x = randn(gen, M, K, dtype=dtype)
    return gen, x, [randn(gen, N, K, scale=K ** -0.5, dtype=dtype) for _ in range(weights)]


# one row to many, one column, odd widths, ends inside of a tile, of a K block and of a vector
SIZES = [(1, 1, 1), (1, 8, 8), (2, 17, 33), (8, 100, 72), (9, 896, 896), (13, 4096, 515), (16, 33, 4096), (17, 16, 16),
         (31, 129, 130), (64, 256, 64), (65, 1, 7), (129, 257, 65), (128, 128, 64), (300, 640, 200), (1, 300, 8192),
         (1000, 1001, 1000), (2048, 1024, 512), (4100, 300, 136), (257, 2304, 4096), (3, 70000, 16)]


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("M,N,K", SIZES)
def test_product_alone(cce, M, N, K, dtype):
    _, x, (w,) = inputs(M, N, K, dtype)
    ref, slack, _, _ = L.linear(x, w)
    y = cce.linear(x, w)
    assert y.dtype == dtype and y.is_contiguous()
    L.within(y, ref, slack, "y")
    L.within(cce.linear(x, w, out_dtype=F32), ref, slack, "y in fp32")


@pytest.mark.parametrize("act", L.ACTS)
@pytest.mark.parametrize("M,N,K", [(1, 300, 200), (16, 129, 136), (33, 100, 72), (129, 257, 65), (700, 520, 264)])
@pytest.mark.parametrize("out,bias,residual", [(None, None, False), (None, F32, True), (F32, BF16, True),
                                               (F32, F16, False)])
def test_epilogue(cce, M, N, K, act, out, bias, residual):
    for dtype in (BF16, F16):
        gen, x, (w,) = inputs(M, N, K, dtype, 1)
        w = w * 2
        b = randn(gen, N, dtype=bias) if bias is not None else None
        r = randn(gen, M, N, dtype=out or dtype) if residual else None
        ref, slack, z, zs = L.linear(x, w, b, r, act)
        y, kept = cce.cce_linear_forward(x, w, b, r, act, out_dtype=out, save=True)
        assert y.dtype == (out or dtype)
        L.within(y, ref, slack, "y")
        if act is None:
            assert kept is None
        else:
            assert kept.dtype == (torch.int16 if dtype == BF16 else dtype)
            L.within_kept(kept, z, zs, "z")
            y2, none = cce.cce_linear_forward(x, w, b, r, act, out_dtype=out)
            assert none is None and torch.equal(y, y2)


@pytest.mark.parametrize("M,N", [(300, 512), (4100, 1001), (40, 264)])
def test_long_sums_in_fp32(cce, M, N):
    """An fp32 result's sum goes on in another accumulator every 1,024 of K: its error is the parts', relative to the norm
    that of K = 1,024 (parts' errors grow together as their sums do, and 8 additions to nearest make 2^-24 each), where one
    accumulator's would be 8 times that.  Twice is allowed."""
    off = []
    for K in (1024, 8192 + 72):
        _, x, (w,) = inputs(M, N, K, BF16, 15)
        ref = x.double() @ w.double().T
        off.append(((cce.linear(x, w, out_dtype=F32) - ref).norm() / ref.norm()).item())
        y, kept = cce.cce_linear_forward(x, w, activation="relu", out_dtype=F32, save=True)
        assert torch.equal(y, cce.linear(x, w, out_dtype=F32).relu())
    assert off[1] < 2 * off[0] + 2.0 ** -23, off


BACKWARD = [(1, 1, 1), (1, 300, 72), (5, 17, 33), (16, 8, 2048), (33, 100, 72), (129, 257, 65), (128, 128, 128),
            (1000, 640, 200), (2048, 896, 896), (4100, 72, 640), (9000, 130, 70), (20000, 8, 8), (256, 4096, 1024)]


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("M,N,K", BACKWARD)
@pytest.mark.parametrize("act,y_type", [(None, None), ("gelu", None), (None, F32), ("silu", F32)])
def test_linear_backward(cce, M, N, K, dtype, act, y_type):
    gen, x, (w,) = inputs(M, N, K, dtype, 2)
    z = randn(gen, M, N, scale=1.5, dtype=dtype) if act else None
    g = randn(gen, M, N, scale=M ** -0.5, dtype=y_type or dtype)
    dz, slack = L.grad_out(g, z if act else g, act)
    (dx, dxs), [(dw, dws)] = L.backward_products([dz], [slack], x, [w], dtype)
    for b_type in (F32, dtype):
        got = cce.cce_linear_backward(g, x, w, z, act, bias_dtype=b_type)
        L.within(got[0], dx, dxs, "dx")
        L.within(got[1], dw, dws, "dw")
        # rows in chains of M / 8 values at most, over groups and blocks: fp32 sums
        db = dz.sum(0)
        assert got[2].dtype == b_type
        L.within(got[2], db, slack.sum(0) + dz.abs().sum(0) * (M / 8 + 300) * 2.0 ** -24, "db")
    # each alone gives the same bits
    for i, need in enumerate(("need_dx", "need_dweight", "need_dbias")):
        only = {k: k == need for k in ("need_dx", "need_dweight", "need_dbias")}
        one = cce.cce_linear_backward(g, x, w, z, act, bias_dtype=dtype, **only)
        assert [t is not None for t in one] == [j == i for j in range(3)]
        L.within(one[i], (dx, dw, dz.sum(0))[i],
                 (dxs, dws, slack.sum(0) + dz.abs().sum(0) * (M / 8 + 300) * 2.0 ** -24)[i], need)


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("act", L.ACTS)
@pytest.mark.parametrize("M,N,K", [(1, 1, 1), (1, 896, 136), (7, 33, 515), (16, 200, 64), (17, 130, 72), (129, 257, 65),
                                   (64, 1000, 896), (2048, 640, 264), (4096, 1024, 512)])
def test_gated_forward(cce, M, N, K, act, dtype):
    _, x, (wg, wu) = inputs(M, N, K, dtype, 3, weights=2)
    wg = wg * 2
    ref, slack, (g, gs), (u, us) = L.gated(x, wg, wu, act)
    y, gate, up = cce.cce_gated_linear_forward(x, wg, wu, act, save=True)
    L.within(y, ref, slack, "y")
    L.within_kept(gate, g, gs, "gate")
    L.within_kept(up, u, us, "up")
    assert torch.equal(y, cce.gated_linear(x, wg, wu, act))


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("act", L.ACTS)
@pytest.mark.parametrize("M,N,K", [(1, 1, 1), (2, 300, 72), (33, 100, 64), (129, 257, 65), (3000, 640, 200),
                                   (2048, 1024, 512)])
def test_gated_backward(cce, M, N, K, act, dtype):
    gen, x, ws = inputs(M, N, K, dtype, 4, weights=2)
    gate, up, g = (randn(gen, M, N, dtype=dtype) for _ in range(3))
    g = g * M ** -0.5
    a, u = L.act64(act, gate.double()), up.double()
    d0, s0 = L.grad_out(g.double() * u, gate, act)
    d1 = g.double() * a
    s0 = s0 + d0.abs() * 2.0 ** -23
    s1 = g.double().abs() * (L.FUNC * gate.double().abs() if act else 0.0) + d1.abs() * 2.0 ** -23
    (dx, dxs), [(dg, dgs), (du, dus)] = L.backward_products([d0, d1], [s0, s1], x, ws, dtype)
    got = cce.cce_gated_linear_backward(g, x, *ws, gate, up, act)
    for t, ref, slack, what in zip(got, (dx, dg, du), (dxs, dgs, dus), ("dx", "dgate_weight", "dup_weight")):
        L.within(t, ref, slack, what)
    for i, need in enumerate(("need_dx", "need_dgate_weight", "need_dup_weight")):
        only = {k: k == need for k in ("need_dx", "need_dgate_weight", "need_dup_weight")}
        one = cce.cce_gated_linear_backward(g, x, *ws, gate, up, act, **only)
        assert [t is not None for t in one] == [j == i for j in range(3)]
        L.within(one[i], (dx, dg, du)[i], (dxs, dgs, dus)[i], need)


def test_kept_words(cce):
    """Both passes through the 16 bits in which pre-activations are kept: rounding,
    subnormals, the range's ends, infinities and NaN."""
    exact = [0.0, 1.0, -1.5, 2.0 ** -30, 2.0 ** -39, -2.0 ** -39, 511 * 2.0 ** -39, 2.0 ** 31, 2.0 ** 31 * (2 - 2.0 ** -9)]
    cases = {v: v for v in exact}
    cases |= {1 + 2.0 ** -10 - 2.0 ** -14: 1.0, -1 - 2.0 ** -10 - 2.0 ** -14: -1 - 2.0 ** -9, 2.0 ** -41: 0.0,
              3 * 2.0 ** -40: 2.0 ** -38, 2.0 ** 31 * (2 - 3 * 2.0 ** -11): 2.0 ** 31 * (2 - 2.0 ** -9), 2.0 ** 32: math.inf, -2.0 ** 40: -math.inf, math.inf: math.inf, -math.inf: -math.inf}
    x = torch.ones(1, 1, device="cuda", dtype=BF16)
    b = torch.tensor(list(cases) + [math.nan], device="cuda")  # z = 0 + bias, in fp32
    w = torch.zeros(len(b), 1, device="cuda", dtype=BF16)
    for rows in (1, 40):
        _, z = cce.cce_linear_forward(x.expand(rows, 1), w, b, activation="relu", save=True)
        want = torch.tensor(list(cases.values()), device="cuda", dtype=torch.float64)
        for row in L.kept(z):
            assert torch.equal(row[:-1], want) and row[-1].isnan()
        small = torch.tensor([v if abs(v) < 2.0 ** 30 else 0.0 for v in cases], device="cuda")  # none at the range's end
        _, zs = cce.cce_linear_forward(x.expand(rows, 1), w[:-1], small, activation="relu", save=True)
        assert torch.equal(L.kept(zs), torch.where(small == 0, 0.0, want).expand(rows, -1))
        # the gate's derivative and the product with it read them
        one = torch.ones(rows, len(b), device="cuda", dtype=BF16)
        fits = [i for i, v in enumerate(cases.values()) if v == torch.tensor(v).bfloat16().item() and abs(v) < 3e38]
        dw = cce.cce_gated_linear_backward(one, x.expand(rows, 1), w, w, z, z, None)[2]
        for i in fits:
            assert dw[i, 0] == rows * torch.tensor(list(cases.values())[i]).bfloat16().item(), list(cases)[i]
        assert dw[-1].isnan().all()


@pytest.mark.parametrize("M,N,K", [(5, 17, 33), (40, 256, 4096), (64, 1000, 896), (129, 257, 65), (300, 640, 200)])
def test_backward_of_kept_words(cce, M, N, K):
    """What a bf16 forward keeps, whole rows on 16 bytes or not and from partial sums, through the backward; columns of
    a wider matrix give the same."""
    gen, x, ws = inputs(M, N, K, BF16, 12, weights=2)
    g = randn(gen, M, N, scale=M ** -0.5, dtype=BF16)

    def apart(words):
        wide = torch.full((M, N + 3), 0x7FFF, dtype=torch.int16, device="cuda")
        wide[:, :N] = words
        return wide[:, :N]

    _, kept = cce.cce_linear_forward(x, ws[0], activation="gelu", save=True)
    _, _, z, zs = L.linear(x, ws[0], act="gelu")
    L.within_kept(kept, z, zs, "z")
    dz, slack = L.grad_out(g, L.kept(kept), "gelu")
    (dx, dxs), [(dw, dws)] = L.backward_products([dz], [slack], x, ws[:1], BF16)
    got = cce.cce_linear_backward(g, x, ws[0], kept, "gelu")
    L.within(got[0], dx, dxs, "dx")
    L.within(got[1], dw, dws, "dw")
    for a, b in zip(got, cce.cce_linear_backward(g, x, ws[0], apart(kept), "gelu")):
        L.within(b, a.double(), 0 * a.double(), "strided")

    _, gate, up = cce.cce_gated_linear_forward(x, *ws, "silu", save=True)
    zg, zu = L.kept(gate), L.kept(up)
    d0, s0 = L.grad_out(g.double() * zu, zg, "silu")
    d1 = g.double() * L.act64("silu", zg)
    s0 = s0 + d0.abs() * 2.0 ** -23
    s1 = g.double().abs() * L.FUNC * zg.abs() + d1.abs() * 2.0 ** -23
    (dx, dxs), dws = L.backward_products([d0, d1], [s0, s1], x, ws, BF16)
    got = cce.cce_gated_linear_backward(g, x, *ws, gate, up, "silu")
    for t, (ref, slack) in zip(got, [(dx, dxs)] + dws):
        L.within(t, ref, slack)
    for a, b in zip(got, cce.cce_gated_linear_backward(g, x, *ws, apart(gate), apart(up), "silu")):
        L.within(b, a.double(), 0 * a.double(), "strided")


def test_no_rows(cce):
    w, w2 = (torch.randn(24, 16, device="cuda", dtype=BF16) for _ in range(2))
    x = torch.empty(3, 0, 16, device="cuda", dtype=BF16, requires_grad=True)
    b = torch.zeros(24, device="cuda", requires_grad=True)
    w.requires_grad_()
    w2.requires_grad_()
    y = cce.linear(x, w, b, activation="gelu")
    assert y.shape == (3, 0, 24)
    y.backward(torch.empty_like(y))
    assert x.grad.shape == x.shape and not w.grad.any() and not b.grad.any()
    w.grad = None
    y = cce.gated_linear(x, w, w2)
    assert y.shape == (3, 0, 24)
    y.backward(torch.empty_like(y))
    assert not w.grad.any() and not w2.grad.any()


@pytest.mark.parametrize("K", [64, 65])
@pytest.mark.parametrize("M", [4, 60])
def test_strides_and_alignment(cce, M, K):
    """Views of larger tensors give the bits of their copies."""
    gen = torch.Generator(device="cuda").manual_seed(5)
    N = 40
    big = randn(gen, 3, M + 2, 2 * K + 16, dtype=BF16)
    wide = randn(gen, N + 3, 3 * K + 5, dtype=BF16)
    res = randn(gen, 3, M + 2, N + 7, dtype=BF16)
    w2 = randn(gen, K, N, dtype=BF16).t()
    views = [big[:, :M, :K], big[:, :M, 8:8 + K], big[:, :M, 3:3 + K], big[:, 1:M + 1, ::2][..., :K],
             big[0, 0, :K].expand(3, M, K), big.transpose(0, 1)[:M, :, :K]]
    weights = [wide[:N, :K], wide[3:, 1:1 + K], w2, wide[0, :K].expand(N, K)]
    for x in views:
        for w in weights:
            r = res[:, 1:M + 1, 2:2 + N] if x.shape[0] == 3 else None
            want = cce.linear(x.contiguous(), w.contiguous(), residual=None if r is None else r.contiguous(),
                              activation="silu")
            assert torch.equal(cce.linear(x, w, residual=r, activation="silu"), want)
            assert torch.equal(cce.gated_linear(x, w, weights[0]),
                               cce.gated_linear(x.contiguous(), w.contiguous(), weights[0].contiguous()))
            z = torch.empty_like(want).normal_(generator=gen)
            for g in (res[:, :M, :N], res[0, 0, :N].expand(3, M, N), res[:, :M, 1:1 + N]):
                g = g if x.shape[0] == 3 else g.transpose(0, 1)
                for act in ("gelu", None):
                    one = cce.cce_linear_backward(g, x, w, z, act)
                    two = cce.cce_linear_backward(g.contiguous(), x.contiguous(), w.contiguous(), z, act)
                    assert all(torch.equal(a, b) for a, b in zip(one, two))


@pytest.mark.parametrize("cols", [1, 3, 4, 7, 33, 130])
def test_strided_fp32_matrices(cce, cols):
    """Residuals and gradients in fp32 at two pitches and off 16 bytes."""
    gen = torch.Generator(device="cuda").manual_seed(12)
    _, x, (w,) = inputs(3 * 20, cols, 24, BF16, 12)
    x = x.view(3, 20, 24)
    big = randn(gen, 3, 22, cols + 6)
    for r in (big[:, :20, :cols], big[:, 1:21, 1:1 + cols], big[:, 2:, 3:3 + cols], big[0, 0, :cols].expand(3, 20, cols),
              big.transpose(0, 1)[:3, :, :cols].expand(3, 3, cols)[:, :1].expand(3, 20, cols)):
        assert torch.equal(cce.linear(x, w, residual=r, out_dtype=F32),
                           cce.linear(x, w, residual=r.contiguous(), out_dtype=F32))
        for a, b in zip(cce.cce_linear_backward(r, x, w), cce.cce_linear_backward(r.contiguous(), x, w)):
            assert torch.equal(a, b)


@pytest.mark.parametrize("M,N,K", [(3, 40, 64), (50, 1001, 72), (20, 256, 4096), (50, 264, 200)])
@pytest.mark.parametrize("out", [None, F32])
def test_residual_in_runs(cce, M, N, K, out):
    """Residuals of every second sequence's rows, of sequences without their last token, and of one row for all, for few
    rows, many and joined partial sums."""
    gen, x, (w,) = inputs(4 * M, N, K, BF16, 14)
    x = x.view(4, M, K)
    big = randn(gen, 8, M + 1, N + 3, dtype=out or BF16)
    for r in (big[::2, :M, :N], big[:4, 1:, 3:], big[::2, ::2, :N][:, :1].expand(4, M, N), big[0, 0, :N].expand(4, M, N),
              big[:4, 0, :N].unsqueeze(1).expand(4, M, N)):
        ref, slack, _, _ = L.linear(x.reshape(-1, K), w, None, r.reshape(-1, N), "silu")
        y = cce.linear(x, w, residual=r, activation="silu", out_dtype=out)
        L.within(y.view(-1, N), ref, slack)
        assert torch.equal(y, cce.linear(x, w, residual=r.contiguous(), activation="silu", out_dtype=out))


def test_what_lies_between_rows_is_not_read(cce):
    """NaN beside the views, in the columns that complete a vector and in the rows behind."""
    for M, N, K in [(3, 20, 20), (40, 50, 36), (300, 130, 100)]:
        full = torch.full((M + 4, K + 28), float("nan"), device="cuda", dtype=BF16)
        wfull = torch.full((N + 4, K + 12), float("nan"), device="cuda", dtype=BF16)
        Kp = (K + 7) // 8 * 8
        x = torch.randn(M, K, device="cuda").bfloat16()
        w = torch.randn(N, K, device="cuda").bfloat16()
        flat_x = torch.full((M, Kp + 8), float("nan"), device="cuda", dtype=BF16)
        flat_w = torch.full((N, Kp + 8), float("nan"), device="cuda", dtype=BF16)
        flat_x[:, :K], flat_w[:, :K] = x, w
        full[:M, :K], wfull[:N, :K] = x, w
        want = cce.linear(x, w)
        assert torch.equal(cce.linear(flat_x[:, :K], flat_w[:, :K]), want)
        assert torch.equal(cce.linear(full[:M, :K], wfull[:N, :K]), want)
        g = torch.randn(M, N, device="cuda").bfloat16()
        for a, b in zip(cce.cce_linear_backward(g, flat_x[:, :K], flat_w[:, :K]), cce.cce_linear_backward(g, x, w)):
            assert torch.equal(a, b)


@pytest.mark.parametrize("M", [5, 40, 600])
def test_infinities_and_nan_stay_in_their_rows_and_columns(cce, M):
    N, K = 136, 72
    _, x, (w, w2) = inputs(M, N, K, BF16, 6, weights=2)
    clean = cce.linear(x, w, activation="silu")
    x2 = x.clone()
    x2[2, 5], x2[3, 7], x2[4, 9] = math.nan, math.inf, -math.inf
    y = cce.linear(x2, w, activation="silu")
    rows = [i for i in range(M) if i not in (2, 3, 4)]
    assert torch.equal(y[rows], clean[rows]) and y[2].isnan().all()
    for a in ("relu", "gelu", "gelu_tanh", "silu"):
        y = cce.linear(x2, w, activation=a)
        up = w[:, 7].float() > 0  # plus infinity stays, minus infinity becomes 0
        down = w[:, 7].float() < 0
        assert (y[3, up] == math.inf).all() and (y[3, down] == 0).all(), a
    g = cce.gated_linear(x2, w, w2)
    assert torch.equal(g[rows], cce.gated_linear(x, w, w2)[rows]) and g[2].isnan().all()
    # a gradient through infinite pre-activations: slope 1 or 0
    z = torch.zeros(M, N, device="cuda", dtype=BF16)
    z[0, 0], z[0, 1], z[0, 2] = math.inf, -math.inf, math.nan
    one = torch.ones(M, N, device="cuda", dtype=BF16)
    for a in ("relu", "gelu", "gelu_tanh", "silu"):
        db = cce.cce_linear_backward(one[:1], x[:1], w, z[:1], a, bias_dtype=F32)[2]
        assert db[0] == 1 and db[1] == 0 and db[2].isnan() and not db[3:].isnan().any(), a


def test_fp16_overflow_is_an_infinity(cce):
    x = torch.full((20, 64), 200.0, device="cuda", dtype=F16)
    w = torch.full((8, 64), 200.0, device="cuda", dtype=F16)
    assert (cce.linear(x, w) == math.inf).all()
    assert (cce.linear(x, w, out_dtype=F32) == 200.0 * 200.0 * 64).all()


@pytest.mark.parametrize("M,N,K", [(3, 40, 24), (70, 136, 65), (600, 256, 128)])
def test_autograd(cce, M, N, K):
    """Gradients of all inputs by autograd are those of the direct calls, and
    those of the formula by differences."""
    gen, x, (w, w2) = inputs(M, N, K, BF16, 7, weights=2)
    b = randn(gen, N)
    r = randn(gen, M, N, dtype=F32)
    g = randn(gen, M, N, dtype=F32)
    leaves = [t.clone().requires_grad_() for t in (x, w, b, r)]
    y = cce.linear(*leaves, activation="gelu_tanh", out_dtype=F32)
    want, z = cce.cce_linear_forward(x, w, b, r, "gelu_tanh", out_dtype=F32, save=True)
    assert torch.equal(y, want)
    grads = torch.autograd.grad(y, leaves, g)
    direct = cce.cce_linear_backward(g, x, w, z, "gelu_tanh", bias_dtype=F32)
    for a, c in zip(grads, direct + (g,)):
        assert torch.equal(a, c)
    # by differences in 64 bits: a direction in each input, error below 1e-5 from a step of 1e-4
    pre = [t.double() for t in (x, w, b, r)]
    for i in range(4):
        d = torch.randn(pre[i].shape, generator=gen, device="cuda", dtype=torch.float64)

        def loss(step):
            t = list(pre)
            t[i] = t[i] + step * d
            return (L.act64("gelu_tanh", t[0] @ t[1].T + t[2]) + t[3]).mul(g.double()).sum()

        slope = (loss(1e-4) - loss(-1e-4)) / 2e-4
        got = (grads[i].double() * d).sum()
        # dz, z and the result are rounded to 16 bits, at random signs: each term off by 3 half steps at most
        terms = (grads[i].double() * d).norm()
        assert abs(got - slope) <= 12 * 3 * 2.0 ** -8 * terms, (i, got.item(), slope.item())
    leaves = [t.clone().requires_grad_() for t in (x, w, w2)]
    y = cce.gated_linear(*leaves)
    gb = g.bfloat16()
    want, gate, up = cce.cce_gated_linear_forward(x, w, w2, save=True)
    assert torch.equal(y, want)
    for a, c in zip(torch.autograd.grad(y, leaves, gb),
                    cce.cce_gated_linear_backward(gb, x, w, w2, gate, up)):
        assert torch.equal(a, c)


def test_autograd_of_some_inputs(cce):
    x, w = torch.randn(6, 16, device="cuda").bfloat16(), torch.randn(8, 16, device="cuda").bfloat16()
    b = torch.randn(8, device="cuda", requires_grad=True)
    r = torch.randn(6, 8, device="cuda").bfloat16().requires_grad_()
    cce.linear(x, w, b, r, "relu").sum().backward()
    assert b.grad is not None and torch.equal(r.grad, torch.ones_like(r))
    r.grad = None
    cce.linear(x, w, residual=r).sum().backward()
    assert torch.equal(r.grad, torch.ones_like(r))
    y = cce.linear(x, w, b.detach(), r)
    y.sum().backward()
    w.requires_grad_()
    cce.gated_linear(x, w, w).sum().backward()  # one weight twice: both gradients add up
    _, gate, up = cce.cce_gated_linear_forward(x, w.detach(), w.detach(), save=True)
    _, dg, du = cce.cce_gated_linear_backward(torch.ones(6, 8, device="cuda").bfloat16(), x, w.detach(), w.detach(), gate, up)
    assert torch.equal(w.grad, dg + du)
    with pytest.raises(RuntimeError, match="not differentiable"):
        v = cce.linear(x.clone().requires_grad_(), w)
        (gw,) = torch.autograd.grad(v.float().square().sum(), w, create_graph=True)
        gw.sum().backward()


def test_repeated_calls_give_the_same_bits(cce):
    for M, N, K in [(16, 896, 896), (100, 896, 4096), (2048, 2304, 896)]:
        gen, x, (w, w2) = inputs(M, N, K, BF16, 8, weights=2)
        g = randn(gen, M, N, dtype=BF16)
        first = None
        for _ in range(3):
            y, gate, up = cce.cce_gated_linear_forward(x, w, w2, save=True)
            now = [y, cce.linear(x, w), *cce.cce_linear_backward(g, x, w),
                   *cce.cce_gated_linear_backward(g, x, w, w2, gate, up)]
            assert first is None or all(torch.equal(a, b) for a, b in zip(first, now))
            first = now


def test_streams_and_graphs(cce):
    """Two streams at once, and a captured step replayed on new values."""
    M, N, K = 300, 264, 136
    gen, x, (w, w2) = inputs(M, N, K, BF16, 9, weights=2)
    want = [cce.linear(x, w, activation="gelu"), cce.gated_linear(x, w, w2)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    out = []
    for i in range(6):
        out.append(cce.cce_linear_forward(x, w, activation="gelu", stream=streams[i % 2])[0])
        out.append(cce.cce_gated_linear_forward(x, w, w2, stream=streams[(i + 1) % 2])[0])
    torch.cuda.synchronize()
    assert all(torch.equal(o, want[i % 2]) for i, o in enumerate(out))

    def step():
        xs = x.detach().requires_grad_()
        ws = w.detach().requires_grad_()
        y = cce.linear(cce.gated_linear(xs, ws, w2), w3, residual=xs)
        return (y, *torch.autograd.grad(y, (xs, ws), torch.ones_like(y)))

    w3 = randn(gen, K, N, scale=N ** -0.5, dtype=BF16)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        captured = step()
    for seed in (10, 11):
        x.copy_(inputs(M, N, K, BF16, seed)[1])
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in captured]
        assert all(torch.equal(a, b) for a, b in zip(got, step()))


def test_large_offsets(cce):
    """Rows behind 2^31 elements, and results there."""
    rows, K, N = 70000, 32768, 8
    x = torch.zeros(rows, K, device="cuda", dtype=BF16)
    x[-3:, :64] = torch.randn(3, 64, device="cuda").bfloat16()
    w = torch.randn(N, K, device="cuda").bfloat16()
    ref, slack, _, _ = L.linear(x[-3:], w)
    L.within(cce.linear(x, w)[-3:], ref, slack, "y")
    g = torch.zeros(rows, N, device="cuda", dtype=BF16)
    g[-1] = 1.0
    dx, dw, _ = cce.cce_linear_backward(g, x, w)
    assert torch.equal(dw, x[-1].expand(N, K)) and not dx[:-1].any()
    L.within(dx[-1:], w.double().sum(0, keepdim=True), w.double().abs().sum(0, keepdim=True) * L.steps(N), "dx")
    del dx, dw
    y = cce.linear(x[:, :64], torch.ones(33000, 64, device="cuda", dtype=BF16))  # 2.3e9 results
    want = x[-3:, :64].double().sum(1, keepdim=True).expand(3, 33000)
    L.within(y[-3:], want, x[-3:, :64].double().abs().sum(1, keepdim=True) * L.steps(64), "y")


def test_refusals(cce):
    x, w = torch.zeros(4, 8, device="cuda", dtype=BF16), torch.zeros(3, 8, device="cuda", dtype=BF16)
    y = torch.zeros(4, 3, device="cuda", dtype=BF16)
    b = torch.zeros(3, device="cuda")
    refused = [
        (lambda: cce.linear(x.float(), w.float()), "bfloat16 or float16"), (lambda: cce.linear(x, w.half()), "weight"),
        (lambda: cce.linear(x, w[:, :7]), "weight"), (lambda: cce.linear(x, w[0]), "weight"),
        (lambda: cce.linear(x, w[:0]), "weight"), (lambda: cce.linear(x, w.cpu()), "weight"),
        (lambda: cce.linear(x[0, 0], w), "last dimension"), (lambda: cce.linear(x[:, :0], w[:, :0]), "last dimension"),
        (lambda: cce.linear(x, w, b[:2]), "bias"), (lambda: cce.linear(x, w, b.double()), "bias"),
        (lambda: cce.linear(x, w, b.cpu()), "bias"), (lambda: cce.linear(x, w, b.expand(3, 3)[:, 0]), "bias"),
        (lambda: cce.linear(x, w, residual=y.float()), "residual"),
        (lambda: cce.linear(x, w, residual=y, out_dtype=F32), "residual"),
        (lambda: cce.linear(x, w, residual=y[:3]), "residual"), (lambda: cce.linear(x, w, residual=b), "residual"),
        (lambda: cce.linear(x, w, out_dtype=F16), "out_dtype"), (lambda: cce.linear(x, w, activation="tanh"), "tanh"),
        (lambda: cce.gated_linear(x, w, w[:2]), "one shape"), (lambda: cce.gated_linear(x, w, w, "swish"), "swish"),
        (lambda: cce.gated_linear(x, w, w.half()), "up_weight"),
        (lambda: cce.cce_linear_backward(y[:3], x, w), "grad_y"), (lambda: cce.cce_linear_backward(y.half(), x, w), "grad_y"),
        (lambda: cce.cce_linear_backward(y, x, w, None, "gelu"), "z"),
        (lambda: cce.cce_linear_backward(y, x, w, y.float(), "gelu"), "z must"),
        (lambda: cce.cce_linear_backward(y.half(), x.half(), w.half(), y.short(), "gelu"), "z must"),
        (lambda: cce.cce_gated_linear_backward(y, x, w, w, y.short(), y), "one type"),
        (lambda: cce.cce_linear_backward(y, x, w, y[:2], "gelu"), "z must"),
        (lambda: cce.cce_linear_backward(y, x, w, bias_dtype=torch.float64), "bias_dtype"),
        (lambda: cce.cce_gated_linear_backward(y, x, w, w, y[:2], y), "gate"),
        (lambda: cce.cce_gated_linear_backward(y, x, w, w, y, y.float()), "up"),
        (lambda: cce.cce_gated_linear_backward(y.float(), x, w, w, y, y), "grad_y"),
    ]
    for call, match in refused:
        with pytest.raises(ValueError, match=match):
            call()


def test_backward_without_an_activation_on_a_fresh_thread(cce):
    """Nothing runs on the autograd engine's thread before the products' own launch."""
    x = torch.randn(300, 64, device="cuda").bfloat16().requires_grad_()
    w = torch.randn(72, 64, device="cuda").bfloat16()
    g = torch.randn(300, 72, device="cuda").bfloat16()
    import threading
    got = []
    y = cce.linear(x, w)

    def run():
        with torch.cuda.device(0):
            got.append(torch.autograd.grad(y, x, g)[0])
    t = threading.Thread(target=run)
    t.start()
    t.join()
    assert torch.equal(got[0], cce.cce_linear_backward(g, x, w)[0])
