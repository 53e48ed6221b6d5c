"""AdamW on the GPU against 64 bits.

Bounds, fixed before any run.  m, v and w are sums of two or three fp32 terms of a
few roundings each (2^-24): at most 8 of them, 2^-21 of the terms' magnitudes.  The
step's size is a quotient with a root: 12 roundings, and with the step counted on the
device expm1 and its argument, 2^-19 of the step at most (t ln beta has half an ulp,
which 1 - beta^t sees at its own size).  A parameter is rounded once more to its type.
8-bit states: the random numbers are the same, so a value is the same multiple of its
scale wherever its unrounded 64-bit value is further from a border of the rounding
than the errors above (of m's terms, which may cancel; of the root itself) and 2^-20
of itself, for the scale and its products, and one step off at most elsewhere; scales
are fp32."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
F8 = torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def cce():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    from tests.conftest import build_library
    build_library()
    import linear_cross_entropy_gb300
    return linear_cross_entropy_gb300


def close(got, ref, magnitude, what, rel=2.0 ** -21):
    fi = torch.finfo(got.dtype)
    slack = rel * magnitude + (2.0 ** -149 if got.dtype == F32 else 0.0)
    tol = (fi.eps / 2 if got.dtype != F32 else 0.0) * (ref.abs() + slack) + slack + fi.smallest_normal * fi.eps / 2
    bad = ~((got.double() - ref).abs() <= tol)
    assert not bad.any(), (what, int(bad.sum()), got[bad][0].item(), ref[bad][0].item())


def reference(w, g, m, v, t, lr, betas, eps, decay, factor=1.0):
    """The new (w, m, v) in 64 bits, and the magnitudes of w's and m's terms."""
    b1, b2 = betas
    g = g.double() * factor
    m1 = b1 * m + (1 - b1) * g
    v1 = b2 * v + (1 - b2) * g * g
    size = lr / (1 - b1 ** t) / ((v1 / (1 - b2 ** t)).sqrt() + eps)
    w1 = w * (1 - lr * decay) - size * m1
    m_terms = b1 * m.abs() + (1 - b1) * g.abs()
    return w1, m1, v1, w.abs() + 8 * size * m_terms, m_terms


HYPER = dict(lr=1e-2, betas=(0.9, 0.99), eps=1e-6, weight_decay=0.1)
SHAPES = {
    "one value": [(1,)],
    "small": [(7,), (128,), (3, 5, 7)],
    "round edges": [(255,), (256,), (257,), (2047,), (2048,), (2049,), (8191,), (8192,), (8193,)],
    "large": [(1000, 5003), (4097, 896), (1,), (65537,)],
    "17 tensors": [(i * 37 + 1,) for i in range(17)],
    "400 tensors": [(i % 301 + 1, 3) for i in range(400)],
    "empty among others": [(0,), (5, 0, 3), (17,), (0, 4), (300, 3)],
}


def make(seed, shapes, p_type, g_type, offset=0):
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def one(s, scale, dtype, positive=False):
        n = math.prod(s)
        flat = scale * torch.randn(n + offset, generator=gen, device="cuda")
        return (flat.square() if positive else flat).to(dtype)[offset:].view(s)

    p = [one(s, 1.0, p_type) for s in shapes]
    g = [one(s, 0.1 * 3.0 ** (i % 5 - 2), g_type) for i, s in enumerate(shapes)]
    m = [one(s, 0.05, F32) for s in shapes]
    v = [one(s, 0.1, F32, True) for s in shapes]
    return p, g, m, v


@pytest.mark.parametrize("p_type,g_type,master", [(BF16, BF16, False), (BF16, BF16, True), (F16, F32, True), (F32, F32, False),
                                                  (F32, BF16, False), (BF16, F32, False), (F16, F16, False),
                                                  (F32, F16, True)])
@pytest.mark.parametrize("shapes", list(SHAPES))
@pytest.mark.parametrize("offset", [0, 1])
def test_update_in_32_bits(cce, shapes, p_type, g_type, master, offset):
    p, g, m, v = make(1, SHAPES[shapes], p_type, g_type, offset)
    masters = [t.float() + 1e-4 for t in p] if master else None
    start = [t.double() for t in (masters or p)]
    refs = [reference(w, b, c.double(), d.double(), 3, HYPER["lr"], HYPER["betas"], HYPER["eps"], HYPER["weight_decay"])
            for w, b, c, d in zip(start, g, m, v)]
    before = [t.clone() for t in g]
    cce.cce_adamw_step(p, g, m, v, 3, masters=masters, **HYPER)
    for i, (w1, m1, v1, w_terms, m_terms) in enumerate(refs):
        close(p[i], w1, w_terms, "param")
        close(m[i], m1, m_terms, "m")
        close(v[i], v1, v1, "v")
        if master:
            close(masters[i], w1, w_terms, "master")
            assert torch.equal(p[i], masters[i].to(p_type))
        assert torch.equal(g[i], before[i])


def test_mixed_kinds_in_one_call(cce):
    sets = [make(i, [(300, 7), (12,)], *types) for i, types in enumerate([(BF16, BF16), (F32, BF16), (F16, F32), (F32, F32)])]
    p, g, m, v = (sum((s[k] for s in sets), []) for k in range(4))
    masters = [t.float().clone() if i % 3 == 0 else None for i, t in enumerate(p)]
    decay = [0.1 * i for i in range(len(p))]
    start = [(w if w is not None else t).double() for w, t in zip(masters, p)]
    refs = [reference(w, b, c.double(), d.double(), 1, 1e-3, (0.9, 0.999), 1e-8, k)
            for w, b, c, d, k in zip(start, g, m, v, decay)]
    cce.cce_adamw_step(p, g, m, v, 1, lr=1e-3, weight_decay=decay, masters=masters)
    for i, (w1, m1, v1, w_terms, m_terms) in enumerate(refs):
        close(p[i], w1, w_terms, "param")
        close(m[i], m1, m_terms, "m")
        close(v[i], v1, v1, "v")


@pytest.mark.parametrize("t", [1, 2, 1000, 100000])
def test_step_and_rate_on_the_device(cce, t):
    p, g, m, v = make(2, [(1000, 3), (5,)], F32, F32)
    q = [[x.clone() for x in y] for y in (p, g, m, v)]
    refs = [reference(a.double(), b, c.double(), d.double(), t, 0.01, (0.9, 0.999), 1e-8, 0.1) for a, b, c, d in zip(p, g, m, v)]
    step, lr = torch.tensor(t, device="cuda"), torch.tensor(0.01, device="cuda")
    cce.cce_adamw_step(p, g, m, v, step, lr=lr, weight_decay=0.1)
    cce.cce_adamw_step(q[0], q[1], q[2], q[3], t, lr=0.01, weight_decay=0.1)
    for i, (w1, _, _, w_terms, _) in enumerate(refs):
        # the rate is rounded to fp32 once more
        close(p[i], w1, w_terms, "step on the device", 2.0 ** -19)
        close(q[0][i], w1, w_terms, "step on the host")


@pytest.mark.parametrize("fraction", [0.3, 2.0, math.inf])
def test_clipping_on_the_way(cce, fraction):
    """The factor is a quotient of the fp32 norm: two roundings more for each gradient."""
    p, g, m, v = make(3, [(500, 5), (4096,)], F32, F32)
    norm = cce.cce_grad_norm(g)
    limit = fraction * norm.item()
    factor = min(1.0, limit / (norm.item() + 1e-6))
    refs = [reference(a.double(), b, c.double(), d.double(), 5, HYPER["lr"], HYPER["betas"], HYPER["eps"],
                      HYPER["weight_decay"], factor) for a, b, c, d in zip(p, g, m, v)]
    cce.cce_adamw_step(p, g, m, v, 5, **HYPER, grad_norm=norm, max_norm=limit)
    for i, (w1, m1, v1, w_terms, m_terms) in enumerate(refs):
        close(p[i], w1, w_terms, "param")
        close(m[i], m1, m_terms, "m")
        close(v[i], v1, v1, "v")
    p, g, _, _ = make(3, [(500, 5), (4096,)], F32, F32)
    state, place = eight_bit_state(cce, p), 0
    refs = [reference(padded(a), padded(b), 0.0 * padded(a), 0.0 * padded(a), 5, HYPER["lr"], HYPER["betas"], HYPER["eps"],
                      HYPER["weight_decay"], factor) for a, b in zip(p, g)]
    cce.cce_adamw8_step(p, g, *state, 5, **HYPER, grad_norm=norm, max_norm=limit)
    for i, (w1, m1, v1, w_terms, m_terms) in enumerate(refs):
        n = p[i].numel()
        words = words_of(0, 5, place, w1.numel())
        place += w1.numel()
        close(p[i].reshape(-1), w1.reshape(-1)[:n], w_terms.reshape(-1)[:n], "param")
        check_held(state[0][i], state[1][i], m1, m_terms, words & 0xFFFF, False, "m")
        check_held(state[2][i], state[3][i], v1.sqrt(), v1.sqrt(), words >> 16, True, "root of v")


def test_norms_that_are_not_finite(cce):
    for norm, limit, want in ((math.nan, 1.0, "nan"), (math.inf, 1.0, "none"), (math.inf, math.inf, "all"), (0.0, 0.0, "all")):
        p, g, m, v = make(4, [(33,)], F32, F32)
        if norm == 0.0:
            g[0].zero_()
        m0, g0 = m[0].clone(), g[0].clone()
        cce.cce_adamw_step(p, g, m, v, 1, lr=0.1, grad_norm=torch.tensor(norm, device="cuda"), max_norm=limit)
        if want == "nan":
            assert m[0].isnan().all() and p[0].isnan().all()
        else:
            f = 1.0 if want == "all" else 0.0
            close(m[0], 0.9 * m0.double() + 0.1 * f * g0.double(), m0.double().abs() + g0.double().abs(), "m")


# -------------------------------------------------------------------- 8 bits
def eight_bit_state(cce, params):
    def codes():
        return [torch.zeros(t.shape, dtype=torch.uint8, device="cuda").view(F8) for t in params]

    def scales():
        return [torch.zeros(cce.adamw_scales(t.numel()), device="cuda") for t in params]
    return [codes(), scales(), codes(), scales()]


def mix(x):
    x = ((x ^ (x >> 16)) * 0x85EBCA6B) & 0xFFFFFFFF
    x = ((x ^ (x >> 13)) * 0xC2B2AE35) & 0xFFFFFFFF
    return x ^ (x >> 16)


def words_of(seed, t, place, n):
    """The random words of n values in whole blocks from `place` on, below 2^32."""
    at = torch.arange(n, device="cuda").view(-1, 256) + place
    return mix(at ^ mix(mix(mix(seed) ^ t) ^ 0))


def padded(t):
    n = t.numel()
    flat = torch.zeros(-(-n // 256) * 256, dtype=torch.float64, device="cuda")
    flat[:n] = t.double().reshape(-1)
    return flat.view(-1, 256)


def held(codes, scales):
    return padded(codes) * scales.double().unsqueeze(1)


def expected(values, terms, words, positive):
    """(lower multiple, upper multiple, scale): both the same where no rounding
    error can cross a border."""
    most = values.abs().amax(1, keepdim=True)
    keep = most >= 2.0 ** -116
    a = torch.where(keep, values.abs() / most * 448, 0.0).nan_to_num(0.0)
    u = words.double() / 65536

    def rounded(a):
        step = torch.ldexp(torch.ones_like(a), (torch.frexp(a).exponent - 4).clamp(min=-9))
        q = (torch.floor(a / step + u) * step).clamp(max=448.0)
        return torch.where((a > 0) & (q < 2.0 ** -9), 2.0 ** -9, q) if positive else q
    off = a * 2.0 ** -20 + torch.where(keep, terms / most * 448, 0.0).nan_to_num(0.0) * 2.0 ** -21
    return rounded((a - off).clamp(min=0.0)), rounded((a + off).clamp(max=448.0)), torch.where(keep, most / 448, 0.0)


def check_held(codes, scales, values, terms, words, positive, what):
    low, high, scale = expected(values, terms, words, positive)
    n = codes.numel()
    got = padded(codes)
    assert (got.abs() >= low - 1e-12).all() and (got.abs() <= high + 1e-12).all(), what
    assert ((low == high) | (high - low <= 32)).all() and ((low != high).sum() <= 4 + 1e-3 * n)
    sign_ok = (got == 0) | (got.sign() == values.sign()) | (values.abs() <= terms * 2.0 ** -21)
    assert sign_ok.all(), what
    assert ((scales.double() - scale.view(-1)).abs() <= 2.0 ** -20 * scale.view(-1)).all(), what


@pytest.mark.parametrize("p_type,g_type,master", [(BF16, BF16, False), (BF16, BF16, True), (F16, F32, False), (F32, F32, False)])
@pytest.mark.parametrize("shapes", list(SHAPES))
@pytest.mark.parametrize("offset", [0, 1])
def test_update_in_8_bits(cce, shapes, p_type, g_type, master, offset):
    p, g, _, _ = make(5, SHAPES[shapes], p_type, g_type, offset)
    masters = [t.float() for t in p] if master else None
    state = eight_bit_state(cce, p)
    seed = 7
    for t in (1, 2) if len(p) > 100 else (1, 2, 3):
        start = [padded(w) for w in (masters or p)]
        refs, place = [], 0
        for i, w in enumerate(start):
            m, r = held(state[0][i], state[1][i]), held(state[2][i], state[3][i])
            refs.append(reference(w, padded(g[i]), m, r * r, t, HYPER["lr"], HYPER["betas"], HYPER["eps"], HYPER["weight_decay"]))
        cce.cce_adamw8_step(p, g, *state, t, masters=masters, seed=seed, **HYPER)
        for i, (w1, m1, v1, w_terms, m_terms) in enumerate(refs):
            n = p[i].numel()
            words = words_of(seed, t, place, w1.numel())
            place += w1.numel()
            close(p[i].reshape(-1), w1.reshape(-1)[:n], w_terms.reshape(-1)[:n], "param")
            check_held(state[0][i], state[1][i], m1, m_terms, words & 0xFFFF, False, "m")
            check_held(state[2][i], state[3][i], v1.sqrt(), v1.sqrt(), words >> 16, True, "root of v")
            if master:
                close(masters[i].reshape(-1), w1.reshape(-1)[:n], w_terms.reshape(-1)[:n], "master")
        g = [x * 0.5 for x in g]


def test_averages_in_8_bits_move(cce):
    """A constant gradient: the averages come near it though each step's change
    is far below a rounding.  v: 1 - 0.999^2000 = 0.865 of g^2, whose root is held with
    steps of at most 1 / 8 and errors that cancel out over 4096 values."""
    p = [torch.zeros(4096, device="cuda")]
    g = [torch.full((4096,), 0.01, device="cuda")]
    g[0][::256] = 0.02  # a larger one in each block: the others are not at the top of the scale
    state = eight_bit_state(cce, p)
    for t in range(1, 2001):
        cce.cce_adamw8_step(p, g, *state, t, lr=0.0, seed=t)
    r = held(state[2][0], state[3][0])[:, 1:]
    want = 0.01 * math.sqrt(1 - 0.999 ** 2000)
    assert abs(r.mean().item() / want - 1) < 0.05
    m = held(state[0][0], state[1][0])[:, 1:]
    assert abs(m.mean().item() / 0.01 - 1) < 0.05


def test_small_values_in_8_bits(cce):
    """Zeros stay zeros, a positive root does not become one, tiny blocks are zeros."""
    p = [torch.zeros(768, device="cuda")]
    g = [torch.zeros(768, device="cuda")]
    g[0][0], g[0][1], g[0][256], g[0][257] = 1.0, 1e-9, 1e-37, 1e-38
    state = eight_bit_state(cce, p)
    cce.cce_adamw8_step(p, g, *state, 1, lr=1e-3)
    r, m = state[2][0].float(), state[0][0].float()
    assert r[0] == 448 and r[1] == 2.0 ** -9 and not r[2:256].any() and not m[512:].any() and not r[512:].any()
    assert state[1][0][1] == 0 and state[1][0][2] == 0 and not m[256:512].any()
    assert p[0][2:256].abs().max() == 0 and p[0].isfinite().all()


def test_nan_and_infinity_in_8_bits_stay_in_their_block(cce):
    p = [torch.zeros(1000, device="cuda")]
    g = [torch.full((1000,), 0.1, device="cuda")]
    g[0][300], g[0][700] = math.nan, math.inf
    state = eight_bit_state(cce, p)
    cce.cce_adamw8_step(p, g, *state, 1, lr=1e-3)
    for codes, scales in ((state[0][0], state[1][0]), (state[2][0], state[3][0])):
        v = held(codes, scales)
        assert v[0].isfinite().all() and v[3].isfinite().all() and v[1].isnan().all() and not v[2].isfinite().any()
    assert p[0][:300].isfinite().all() and p[0][301:700].isfinite().all() and p[0][300].isnan()


# ------------------------------------------------------------------ layout
def test_layouts(cce):
    """Parameters of any dense order; gradients of any strides."""
    gen = torch.Generator(device="cuda").manual_seed(6)

    def rnd(*s):
        return torch.randn(s, generator=gen, device="cuda")
    cases = [(rnd(6, 8).t(), rnd(8, 6)), (rnd(8, 6), rnd(6, 8).t()), (rnd(2, 3, 4, 5).permute(0, 2, 3, 1), rnd(2, 4, 5, 3)),
             (rnd(9, 7), rnd(7).expand(9, 7)), (rnd(9, 7), rnd(9, 14)[:, ::2]), (rnd(), rnd()),
             (rnd(5), torch._neg_view(rnd(5)))]
    for p, g in cases:
        m, v = torch.zeros_like(p), torch.zeros_like(p)
        w1, m1, v1, wt, mt = reference(p.double(), g, m.double(), v.double(), 1, 1e-2, (0.9, 0.999), 1e-8, 0.01)
        version = p._version
        cce.cce_adamw_step([p], [g], [m], [v], 1, lr=1e-2)
        assert p._version > version
        close(p, w1, wt, "param")
        close(m, m1, mt, "m")
        close(v, v1, v1, "v")


def test_refusals(cce):
    p, g, m, v = ([torch.zeros(8, 4, device="cuda")] for _ in range(4))
    s8 = eight_bit_state(cce, p)

    def step(*args, **kw):
        return lambda: cce.cce_adamw_step(*args, **({"lr": 1e-3} | kw))

    def step8(*args, **kw):
        return lambda: cce.cce_adamw8_step(*args, **({"lr": 1e-3} | kw))
    half = [torch.zeros(8, 4, device="cuda", dtype=BF16)]
    for call in [step(p, [], m, v, 1), step(p, g, m, [], 1), step(p, g, m, v, 0), step(p, g, m, v, -3), step(p, g, half, v, 1),
                 step(p, g, m, half, 1), step(p, g, m, v, 1, masters=half), step(p, g, m, v, 1, masters=[None, None]),
                 step(p, g, m, v, 1, weight_decay=[0.1, 0.1]), step(p, g, m, v, 1, max_norm=1.0),
                 step(p, g, m, v, 1, grad_norm=torch.ones((), device="cuda")),
                 step(p, g, m, v, 1, grad_norm=torch.ones((), device="cuda"), max_norm=math.nan),
                 step(p, g, m, v, 1, grad_norm=torch.ones(2, device="cuda"), max_norm=1.0),
                 step(p, g, m, v, 1, grad_norm=torch.ones((), device="cuda", dtype=torch.float64), max_norm=1.0),
                 step(p, g, m, v, 1, grad_norm=torch.ones(()), max_norm=1.0),
                 step(p, g, m, v, torch.ones((), device="cuda")), step(p, g, m, v, torch.ones((), dtype=torch.int64)),
                 step(p, g, m, v, 1, lr=torch.ones((), device="cuda", dtype=torch.float64)),
                 step(p, [g[0].t()], m, v, 1), step(p, [g[0].double()], m, v, 1), step([p[0].double()], g, m, v, 1),
                 step(p, g, [m[0].t().contiguous().t()], v, 1), step(p, [g[0].cpu()], m, v, 1), step([p[0].cpu()], g, m, v, 1),
                 step([torch.zeros(8, 8, device="cuda")[:, :4]], g, m, v, 1), step([p[0][:1].expand(8, 4)], g, m, v, 1),
                 step([torch._neg_view(p[0])], g, m, v, 1), step(p, [g[0].to_sparse()], m, v, 1),
                 step8(p, g, m, s8[1], s8[2], s8[3], 1), step8(p, g, s8[0], [], s8[2], s8[3], 1),
                 step8(p, g, s8[0], [s8[1][0][:0]], s8[2], s8[3], 1), step8(p, g, s8[0], [s8[1][0].double()], s8[2], s8[3], 1)]:
        with pytest.raises(ValueError):
            call()
    for call in [step(p, p, m, v, 1), step(p + p, g + g, m + m, v + v, 1), step(p, g, m, m, 1), step(p, g, m, v, 1, masters=p),
                 step(p, g, m, v, 1, betas=(1.0, 0.9)), step(p, g, m, v, 1, betas=(0.9, -0.1)), step(p, g, m, v, 1, lr=-1.0),
                 step(p, g, m, v, 1, lr=math.nan), step(p, g, m, v, 1, eps=-1.0), step(p, g, m, v, 1, weight_decay=-0.1)]:
        with pytest.raises(cce.CCEError):
            call()
    cce.cce_adamw_step([], [], [], [], 1, lr=1e-3)
    assert not p[0].any() and not m[0].any()


# --------------------------------------------------------------- optimiser
@pytest.mark.parametrize("bits", [8, 32])
def test_optimiser(cce, bits):
    """The class makes the direct calls' updates, also after its state went
    through a state_dict."""
    def params():
        torch.manual_seed(1)
        return [torch.nn.Parameter(torch.randn(s, device="cuda").to(d)) for s, d in (((64, 128), BF16), ((128,), F32), ((96, 50), F16))]

    def grads(ps, t):
        torch.manual_seed(10 + t)
        for p in ps:
            p.grad = torch.randn(p.shape, device="cuda").to(p.dtype)
    a, b = params(), params()
    kw = dict(lr=1e-2, state_bits=bits, master_weights=True, min_8bit_size=1000, seed=3)
    one, two = cce.AdamW(a, **kw), cce.AdamW(b, **kw)
    for t in range(4):
        if t == 2:  # through a checkpoint
            saved = two.state_dict()
            two = cce.AdamW(b, **kw)
            two.load_state_dict(saved)
        grads(a, t)
        grads(b, t)
        if t == 1:
            a[1].grad = b[1].grad = None
        norm = cce.cce_grad_norm([p.grad for p in a if p.grad is not None])
        one.step(grad_norm=norm, max_norm=1.0)
        two.step(grad_norm=norm, max_norm=1.0)
        for p, q in zip(a, b):
            assert torch.equal(p, q)
            for k, v in one.state[p].items():
                w = two.state[q][k]
                assert torch.equal(v.view(torch.uint8), w.view(torch.uint8)) if isinstance(v, torch.Tensor) else v == w
    assert one.state[a[0]]["step"] == 4 and one.state[a[1]]["step"] == 3
    assert one.state[a[0]]["exp_avg"].dtype == (F8 if bits == 8 else F32) and one.state[a[0]]["master"].dtype == F32
    assert "master" not in one.state[a[1]] and one.state[a[1]]["exp_avg"].dtype == F32


@pytest.mark.parametrize("bits", [8, 32])
def test_captured_steps(cce, bits):
    def make_one(capturable):
        torch.manual_seed(2)
        p = [torch.nn.Parameter(torch.randn(5000, device="cuda").bfloat16()), torch.nn.Parameter(torch.randn(70, device="cuda"))]
        for q in p:
            q.grad = torch.randn(q.shape, device="cuda").to(q.dtype)
        return p, cce.AdamW(p, lr=1e-2, state_bits=bits, capturable=capturable)
    p, opt = make_one(True)
    q, plain = make_one(False)
    opt.step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        opt.step()
    for _ in range(3):
        graph.replay()
    for _ in range(4):
        plain.step()
    assert opt.state[p[0]]["step"].item() == 4 and opt.state[p[0]]["step"] is opt.state[p[1]]["step"]
    for a, b in zip(p, q):
        # 1 - beta^t comes from expm1 there: 2^-19 of a step of 1e-2 each, and a rounding of a bf16 parameter
        fi = torch.finfo(a.dtype)
        assert ((a - b).abs().double() <= 4 * (1e-2 * 2.0 ** -18 + fi.eps * b.abs().double())).all()


def test_two_streams_and_repeats(cce):
    sets = []
    for _ in range(2):
        p, g, _, _ = make(8, [(5000, 9), (77,)], BF16, BF16)
        sets.append((p, g, eight_bit_state(cce, p)))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for t in range(1, 6):
        for (p, g, s), stream in zip(sets, streams):
            cce.cce_adamw8_step(p, g, *s, t, lr=1e-2, stream=stream)
    torch.cuda.synchronize()
    (a, _, sa), (b, _, sb) = sets
    for x, y in zip(a + sum(sa, []), b + sum(sb, [])):
        assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))
