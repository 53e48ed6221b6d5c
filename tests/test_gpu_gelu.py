"""gelu keeps its relative accuracy where the normal distribution function vanishes.

Bound, fixed before any run: gelu(z) = z Phi(z), for negative z with
Phi = e^(-z^2 / 2) P / Q.  The exponent's two products and its constant are rounded, at
most 3 * 2^-24 of z^2 / 2 in all, and as much of Phi: z^2 2^-23.  P / Q is within
4.9e-7, 4.1 * 2^-23, of its value, and with 4 roundings each of P and Q, whose terms are
positive, 4 of products, 2 ulp each of the power of two and the reciprocal and one of the
last product there are 16 * 2^-23.  Values below 2^-126 may count as 0."""
import math

import pytest
import torch

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


def phi(z):
    return 0.5 * torch.special.erfc(-z / math.sqrt(2))


def gate_slack(z):
    return phi(z) * (z * z + 16) * 2.0 ** -23 + 2.0 ** -126


def half_step(ref, dtype):
    fi = torch.finfo(dtype)
    return ref.abs() * (fi.eps / 2) + fi.smallest_normal * fi.eps / 2


def values(lo, hi):
    z = torch.linspace(lo, hi, 4000, device="cuda")
    return torch.cat([z, z.bfloat16().float(), torch.tensor([0.0, -0.0, 1e-30, -1e-30], device="cuda")])


def pre_activations(rows, z, dtype):
    """x, weight and bias whose z is the bias."""
    return (torch.zeros(rows, 8, device="cuda", dtype=dtype), torch.zeros(z.numel(), 8, device="cuda", dtype=dtype), z)


@pytest.mark.parametrize("rows", [1, 40])
@pytest.mark.parametrize("dtype,out", [(BF16, F32), (F16, F32), (BF16, BF16), (F16, F16)])
def test_tail(cce, rows, dtype, out):
    for lo, hi in ((-6, -3), (-16, 0), (0, 16)):
        z = values(lo, hi)
        y = cce.linear(*pre_activations(rows, z, dtype), activation="gelu", out_dtype=out)
        ref = z.double() * phi(z.double())
        slack = z.double().abs() * gate_slack(z.double()) + ref.abs() * 2.0 ** -24
        tol = slack + (half_step(ref.abs() + slack, out) if out != F32 else 2.0 ** -149)
        bad = ~((y.double() - ref).abs() <= tol)
        assert not bad.any(), (z[bad.any(0)][:4].tolist(), y[bad][:4].tolist(), ref[bad.any(0)][:4].tolist())


@pytest.mark.parametrize("rows", [1, 40])
def test_splits_join_the_same_function(cce, rows):
    """From partial sums of a K in several parts, and in one, the same bits."""
    z = values(-8, 8)[:1000].contiguous()
    short = cce.linear(*pre_activations(rows, z, BF16), activation="gelu", out_dtype=F32)
    long = cce.linear(torch.zeros(rows, 9000, device="cuda", dtype=BF16),
                      torch.zeros(z.numel(), 9000, device="cuda", dtype=BF16), z, activation="gelu", out_dtype=F32)
    assert torch.equal(short, long)


def test_backward_of_a_gated_layer_reads_the_same_function(cce):
    """dup = grad act(gate): one row, one x of 1, so that dup_weight is dup, rounded to bf16 once."""
    z = values(-13, 13).bfloat16()
    one = torch.ones(1, 1, device="cuda", dtype=BF16)
    w = torch.zeros(z.numel(), 1, device="cuda", dtype=BF16)
    g = torch.ones(1, z.numel(), device="cuda", dtype=BF16)
    up = torch.ones(1, z.numel(), device="cuda", dtype=BF16)
    _, dgate, dup = cce.cce_gated_linear_backward(g, one, w, w, z.view(1, -1), up, "gelu")
    d = z.double()
    ref = d * phi(d)
    slack = d.abs() * gate_slack(d) + ref.abs() * 2.0 ** -24
    # once to the products' 16 bits, and the product with 1 is exact
    assert ((dup.view(-1).double() - ref).abs() <= slack + half_step(ref.abs() + slack, BF16)).all()
    y = cce.linear(*pre_activations(1, z.float(), BF16), activation="gelu")
    assert torch.equal(dup.view(-1), y.view(-1))
    # the slope's two terms: the gate, and z times the density (three roundings and the exponent's)
    density = torch.exp(-d * d / 2) / math.sqrt(2 * math.pi)
    slope = phi(d) + d * density
    slack = gate_slack(d) + (d * density).abs() * (d * d + 8) * 2.0 ** -23 + slope.abs() * 2.0 ** -24 + d.abs() * 2.0 ** -126
    assert ((dgate.view(-1).double() - slope).abs() <= slack + half_step(slope.abs() + slack, BF16)).all()
