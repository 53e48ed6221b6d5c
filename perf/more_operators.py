"""Cases of the operators in front of the loss head and behind its gradients:
linear layers with a fused epilogue, gated linear layers, and AdamW.

The classifier reads hidden states that a dense transform or a feed-forward
block has produced (a prediction head is such a transform with a residual), and
a training step ends with the update of all parameters.  Each case is one call
(or one forward and backward) of such an operator, in its plain form
(elementary torch operations in 32 bits) or, with `own` set, through
linear_cross_entropy_gb300.
"""
import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
BYTES = {"bf16": 2, "fp16": 2, "fp32": 4}
CLIP_EPS = 1e-6  # added to the gradients' norm before the division
BLOCK = 256  # values that share a scale in 8-bit states
TOP = 448.0  # the largest e4m3 value
TINY = 2.0 ** -116  # a block whose largest magnitude is below is held as zeros


# ------------------------------------------------------------------- cases
def _linear_case(name, pass_, batch, seq, dim, out, x="bf16", y=None, act="none", bias="", residual=False, shift=False):
    return {"name": name, "op": "linear", "pass": pass_, "batch": batch, "seq": seq, "dim": dim, "out": out, "x": x,
            "y": y or x, "act": act, "bias": bias, "residual": residual, "shift": shift}


def _gated_case(name, pass_, batch, seq, dim, out, x="bf16", act="silu", shift=False):
    return {"name": name, "op": "gated", "pass": pass_, "batch": batch, "seq": seq, "dim": dim, "out": out, "x": x,
            "act": act, "shift": shift}


def _adamw_case(name, layers, dim, vocab, p="bf16", g="bf16", bits=32, master=False, clip=True, t=100):
    return {"name": name, "op": "adamw", "layers": layers, "dim": dim, "vocab": vocab, "p": p, "g": g, "bits": bits,
            "master": master, "clip": clip, "t": t}


def listed():
    return [
        # decoding one token: the transform in front of the classifier, all latency
        _linear_case("linear 1 token", "forward", 1, 1, 896, 896, act="gelu", bias="bf16"),
        # decoding a small odd batch through a prediction head: y = x + silu(W x + b)
        _linear_case("linear 13 tokens", "forward", 13, 1, 4096, 4096, x="fp16", act="silu", bias="fp16", residual=True),
        # every token but the last of each sequence, an odd width, a 32-bit residual stream
        _linear_case("linear odd", "forward", 7, 147, 1000, 1001, y="fp32", act="relu", bias="fp32", residual=True, shift=True),
        # the backward of a Qwen2.5-0.5B-shaped transform
        _linear_case("linear backward", "backward", 1, 4096, 896, 896, act="gelu_tanh", bias="fp32"),
        # the projection back to a Gemma-2-2B-shaped residual stream, trained
        _linear_case("linear step", "step", 4, 2048, 9216, 2304, residual=True),
        # the first product of a feed-forward block over the long-context batch of 65,536 tokens
        _linear_case("linear long", "forward", 1, 65536, 2048, 8192, act="gelu", bias="bf16"),
        # decoding one token through a gated block
        _gated_case("gated 1 token", "forward", 1, 1, 896, 4864),
        # the forward of a Gemma-2-2B-shaped batch
        _gated_case("gated forward", "forward", 4, 2048, 2304, 9216, act="gelu_tanh"),
        # a training step of a Qwen2.5-0.5B-shaped batch
        _gated_case("gated step", "step", 1, 4096, 896, 4864),
        # the head alone being trained at its smallest size
        _adamw_case("adamw tiny head", 0, 128, 4096),
        # a Qwen2.5-0.5B-shaped head, states in 8 bits
        _adamw_case("adamw 8-bit head", 0, 896, 151936, bits=8),
        # a whole 24-layer model with 32-bit master weights
        _adamw_case("adamw model", 24, 896, 151936, master=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def _width(rng, lo, hi):
    """An odd multiple of 1, 8, 128 or 512."""
    step = rng.choice((1, 8, 8, 128, 512))
    return step * (_log(rng, max(1, lo // step), max(1, (hi - step) // step)) | 1)


def draw(rng):
    case = _drawn(rng)
    del case["name"]
    return case


def _drawn(rng):
    if rng.random() < 0.3:
        p = rng.choice(("bf16", "bf16", "fp16", "fp32"))
        return _adamw_case("", rng.choice((0, 0, _log(rng, 1, 24))), _width(rng, 64, 896), _log(rng, 1000, 131072), p=p,
                           g=rng.choice((p, "fp32")), bits=rng.choice((8, 32)), master=p != "fp32" and rng.random() < 0.5,
                           clip=rng.random() < 0.5, t=_log(rng, 1, 10000))
    dim, out = _width(rng, 64, 10240), _width(rng, 64, 10240)
    pass_ = rng.choice(("forward", "forward", "backward", "step"))
    gated = rng.random() < 0.4
    products = {"forward": 1, "backward": 2, "step": 3}[pass_] * (2 if gated else 1)
    rows = _log(rng, 1, min(65536, 65536 * 2048 * 8192 // (dim * out * products)))
    batch = min(rows, rng.choice((1, 2, 7, 16)))
    seq = max(1, rows // batch)
    x = rng.choice(("bf16", "bf16", "fp16"))
    shift = seq > 1 and rng.random() < 0.25
    if gated:
        return _gated_case("", pass_, batch, seq, dim, out, x=x, act=rng.choice(("silu", "gelu", "gelu_tanh", "relu")),
                           shift=shift)
    # a step rounds what its backward reads to 16 bits: a 32-bit bias is for the other passes
    bias = rng.choice(("", x, x if pass_ == "step" else "fp32"))
    return _linear_case("", pass_, batch, seq, dim, out, x=x, y=rng.choice((x, x, "fp32")),
                        act=rng.choice(("none", "relu", "gelu", "gelu_tanh", "silu")), bias=bias,
                        residual=rng.random() < 0.5, shift=shift)


def _rows(case):
    return case["batch"] * (case["seq"] - 1 if case["shift"] else case["seq"])


def _shapes(case):
    """The parameters of a decoder of that width (attention, gated MLP, norms) and of its head."""
    d = case["dim"]
    layer = [(d, d)] * 4 + [(d,)] * 3 + [(4 * d, d)] * 2 + [(d, 4 * d)] + [(d,)] * 2
    return layer * case["layers"] + [(d,), (d,), (case["vocab"], d)]


# ------------------------------------------------------------------ inputs
def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def randn(*shape):
        return torch.randn(shape, generator=gen, device="cuda")

    return _prepare_adamw(case, seed, gen, randn) if case["op"] == "adamw" else _prepare_linear(case, randn)


def _cut(case, t):
    return t[:, :-1] if case["shift"] else t


def _prepare_linear(case, randn):
    b, s, d, n = case["batch"], case["seq"], case["dim"], case["out"]
    kind = TYPES[case["x"]]
    # normalised hidden states, a few channels of which stand out
    scale = torch.exp(0.2 * randn(d))
    scale[::97] *= 4.0
    x = _cut(case, (randn(b, s, d) * scale).to(kind))
    state = {"case": case, "x": x}
    names = ("wg", "wu") if case["op"] == "gated" else ("w",)
    for k in names:
        state[k] = (randn(n, d) / math.sqrt(d)).to(kind)
    if case["op"] == "linear":
        if case["bias"]:
            state["b"] = (0.2 * randn(n)).to(TYPES[case["bias"]])
        if case["residual"]:
            state["r"] = _cut(case, randn(b, s, n).to(TYPES[case["y"]]))
    if case["pass"] != "forward":
        state["dy"] = _cut(case, (1e-2 * randn(b, s, n)).to(TYPES[case.get("y", case["x"])]))
    if case["pass"] == "backward":  # what the forward pass left
        for k, z in zip(names, _products(state, names)):
            state["z" + k] = z.to(kind)
        state.pop("r", None)
    if case["pass"] == "step":
        for k in ("x", "w", "wg", "wu", "b", "r"):
            if k in state:
                state[k] = state[k].detach().requires_grad_()
    return state


@torch.no_grad()
def _products(state, names):
    x = state["x"].float()
    bias = state["b"].float() if "b" in state else 0.0
    return [x @ state[k].float().T + bias for k in names]


def _prepare_adamw(case, seed, gen, randn):
    shapes = _shapes(case)
    sizes = [math.prod(s) for s in shapes]
    # one buffer for each kind of value, where tensors start on whole blocks
    padded = [-(-n // BLOCK) * BLOCK for n in sizes]
    total = sum(padded)
    used = torch.ones(total, dtype=torch.bool, device="cuda")
    for part, n in zip(used.split(padded), sizes):
        part[n:] = False

    def flat(std):
        return (randn(total) * std).mul_(used)

    weight = flat(0.02)
    # gradients whose size differs from one part of the model to the next
    level = torch.exp(randn(total // BLOCK).repeat_interleave(BLOCK)).mul_(1e-3)
    grad = flat(level)
    first, root = flat(level * 0.3), (randn(total).abs_().add_(0.3)).mul_(level).mul_(used)
    state = {"case": case, "sizes": sizes, "padded": padded, "seed": seed % 1000003,
             "p": weight.to(TYPES[case["p"]]), "g": grad.to(TYPES[case["g"]])}
    if case["master"]:
        state["master"] = weight
    if case["clip"]:
        state["norm"] = state["g"].float().square().sum().sqrt()
        state["max_norm"] = 0.5 * float(state["norm"])
    if case["bits"] == 32:
        state["m"], state["v"] = first, root.square_()
    else:
        state["m"], state["ms"] = _held(first)
        state["r"], state["rs"] = _held(root)
    state["lists"] = {k: _views(state, k, shapes) for k in ("p", "g", "master", "m", "v", "r") if k in state}
    for k in ("ms", "rs"):
        if k in state:
            state["lists"][k] = list(state[k].split([q // BLOCK for q in padded]))
    return state


def _views(state, k, shapes):
    parts = state[k].split(state["padded"])
    return [t[:n].view(s) for t, n, s in zip(parts, state["sizes"], shapes)]


def _held(values):
    """8-bit values, to nearest, and a scale for each block."""
    blocks = values.view(-1, BLOCK)
    scale = blocks.abs().amax(1) / TOP
    return (blocks / scale.clamp(min=1e-30).unsqueeze(1)).to(torch.float8_e4m3fn).view(-1), scale


# -------------------------------------------------------------- plain forms
def _activation(act, z):
    if act == "relu":
        return z.clamp(min=0.0)
    if act == "gelu":
        return 0.5 * z * (1.0 + torch.erf(z * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return 0.5 * z * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (z + 0.044715 * z ** 3)))
    return z / (1.0 + torch.exp(-z)) if act == "silu" else z


def _slope(act, z):
    """The derivative of the activation."""
    if act == "relu":
        return (z > 0.0).to(z.dtype)
    if act == "gelu":
        return 0.5 * (1.0 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) / math.sqrt(2.0 * math.pi)
    if act == "gelu_tanh":
        c = math.sqrt(2.0 / math.pi)
        t = torch.tanh(c * (z + 0.044715 * z ** 3))
        return 0.5 * (1.0 + t) + 0.5 * z * (1.0 - t * t) * c * (1.0 + 3 * 0.044715 * z * z)
    if act == "silu":
        s = 1.0 / (1.0 + torch.exp(-z))
        return s * (1.0 + z * (1.0 - s))
    return torch.ones_like(z)


def _plain_linear(state):
    case = state["case"]
    x = state["x"].float()
    kind = state["x"].dtype
    out = {}
    z = state["zw"].float() if "zw" in state else _products(state, ("w",))[0]
    if case["pass"] != "backward":
        y = _activation(case["act"], z)
        out["y"] = (y + state["r"].float() if "r" in state else y).to(TYPES[case["y"]])
    if case["pass"] != "forward":
        dz = state["dy"].float() * _slope(case["act"], z)
        flat = dz.reshape(-1, case["out"])
        out["dx"] = (dz @ state["w"].float()).to(kind)
        out["dw"] = (flat.T @ x.reshape(-1, case["dim"])).to(kind)
        if "b" in state:
            out["db"] = flat.sum(0).to(state["b"].dtype)
    return out


def _plain_gated(state):
    case = state["case"]
    x = state["x"].float()
    kind = state["x"].dtype
    out = {}
    gate, up = (state["zwg"].float(), state["zwu"].float()) if "zwg" in state else _products(state, ("wg", "wu"))
    a = _activation(case["act"], gate)
    if case["pass"] != "backward":
        out["y"] = (a * up).to(kind)
    if case["pass"] != "forward":
        dy = state["dy"].float()
        dgate, dup = dy * up * _slope(case["act"], gate), dy * a
        rows = x.reshape(-1, case["dim"])
        out["dx"] = (dgate @ state["wg"].float() + dup @ state["wu"].float()).to(kind)
        out["dwg"] = (dgate.reshape(-1, case["out"]).T @ rows).to(kind)
        out["dwu"] = (dup.reshape(-1, case["out"]).T @ rows).to(kind)
    return out


LR, BETA1, BETA2, EPS, DECAY = 1e-3, 0.9, 0.999, 1e-8, 0.1


def _mix(x):
    """The finaliser of MurmurHash3 on 32-bit words (held in 64 bits)."""
    low = 0xFFFFFFFF
    x = ((x ^ (x >> 16)) * 0x85EBCA6B) & low
    x = ((x ^ (x >> 13)) * 0xC2B2AE35) & low
    return x ^ (x >> 16)


def _random_words(state, n):
    """32 random bits for each value, from the seed, the step and the value's place."""
    key = _mix(_mix(state["seed"] & 0xFFFFFFFF) ^ (state["case"]["t"] & 0xFFFFFFFF))
    at = torch.arange(n, device="cuda")
    return _mix((at & 0xFFFFFFFF) ^ _mix(key ^ (at >> 32)))


def _round8(values, words, positive):
    """Values rounded at random to e4m3 (up with the distance from the lower
    neighbour as probability), and their blocks' scales.  Positive ones do not
    become 0."""
    blocks = values.view(-1, BLOCK)
    most = blocks.abs().amax(1, keepdim=True)
    kept = ~(most < TINY)
    a = torch.where(kept, blocks.abs() * (TOP / most), 0.0).clamp(max=TOP)
    # a's step: 2^-3 of its power of two, 2^-9 at least
    step = torch.ldexp(torch.ones_like(a), (torch.frexp(a).exponent - 4).clamp(min=-9))
    q = torch.floor(a / step + words.view(-1, BLOCK).to(a.dtype) * 2.0 ** -16) * step
    q = q.clamp(max=TOP)
    if positive:
        q = torch.where((a > 0.0) & (q < 2.0 ** -9), 2.0 ** -9, q)
    q = torch.where(blocks < 0.0, -q, q)
    return q.to(torch.float32).to(torch.float8_e4m3fn).view(-1), torch.where(kept, most / TOP, 0.0).view(-1)


def _plain_adamw(state):
    new = _adamw(state)
    return {k: state[k].copy_(v) for k, v in new.items()}


def _adamw(state):
    """The new values of the state's buffers."""
    case = state["case"]
    g = state["g"].float()
    if case["clip"]:
        g = g * (state["max_norm"] / (state["norm"] + CLIP_EPS)).clamp(max=1.0)
    weight = (state["master"] if case["master"] else state["p"]).float()
    if case["bits"] == 32:
        m, v = state["m"].float(), state["v"].float()
    else:
        m = (state["m"].float().view(-1, BLOCK) * state["ms"].float().unsqueeze(1)).view(-1)
        v = (state["r"].float().view(-1, BLOCK) * state["rs"].float().unsqueeze(1)).view(-1).square()
    m = BETA1 * m + (1.0 - BETA1) * g
    v = BETA2 * v + (1.0 - BETA2) * g * g
    c1, c2 = 1.0 - BETA1 ** case["t"], 1.0 - BETA2 ** case["t"]
    root = v.sqrt()
    weight = weight * (1.0 - LR * DECAY) - LR / c1 * m / (root / math.sqrt(c2) + EPS)
    out = {"p": weight}
    if case["master"]:
        out["master"] = weight
    if case["bits"] == 32:
        return out | {"m": m, "v": v}
    words = _random_words(state, m.numel())
    out["m"], out["ms"] = _round8(m, words & 0xFFFF, False)
    out["r"], out["rs"] = _round8(root, words >> 16, True)
    return out


@torch.no_grad()
def _run_plain(state):
    return {"linear": _plain_linear, "gated": _plain_gated, "adamw": _plain_adamw}[state["case"]["op"]](state)


# ----------------------------------------------------------- the operators
def _own_linear(cce, state):
    case = state["case"]
    act = None if case["act"] == "none" else case["act"]
    w, b = state["w"], state.get("b")
    if case["pass"] == "backward":
        z = state["zw"] if act else None
        grads = cce.cce_linear_backward(state["dy"], state["x"], w, z, act, need_dbias=b is not None,
                                        bias_dtype=b.dtype if b is not None else None)
        return {k: g for k, g in zip(("dx", "dw", "db"), grads) if g is not None}
    y = cce.linear(state["x"], w, b, residual=state.get("r"), activation=act, out_dtype=TYPES[case["y"]])
    if case["pass"] == "forward":
        return {"y": y}
    names = [k for k in ("x", "w", "b") if k in state]
    return {"y": y.detach()} | dict(zip(["d" + k for k in names],
                                        torch.autograd.grad(y, [state[k] for k in names], state["dy"])))


def _own_gated(cce, state):
    case = state["case"]
    x, wg, wu = state["x"], state["wg"], state["wu"]
    if case["pass"] == "backward":
        grads = cce.cce_gated_linear_backward(state["dy"], x, wg, wu, state["zwg"], state["zwu"], case["act"])
        return dict(zip(("dx", "dwg", "dwu"), grads))
    y = cce.gated_linear(x, wg, wu, case["act"])
    if case["pass"] == "forward":
        return {"y": y}
    return {"y": y.detach()} | dict(zip(("dx", "dwg", "dwu"), torch.autograd.grad(y, (x, wg, wu), state["dy"])))


def _own_adamw(cce, state):
    case, t = state["case"], state["lists"]
    more = {"lr": LR, "betas": (BETA1, BETA2), "eps": EPS, "weight_decay": DECAY, "masters": t.get("master")}
    if case["clip"]:
        more |= {"grad_norm": state["norm"], "max_norm": state["max_norm"]}
    if case["bits"] == 32:
        cce.cce_adamw_step(t["p"], t["g"], t["m"], t["v"], case["t"], **more)
    else:
        cce.cce_adamw8_step(t["p"], t["g"], t["m"], t["ms"], t["r"], t["rs"], case["t"], seed=state["seed"], **more)
    return {k: state[k] for k in ("p", "master", "m", "v", "ms", "r", "rs") if k in state}


def _run_own(state):
    import linear_cross_entropy_gb300 as cce

    return {"linear": _own_linear, "gated": _own_gated, "adamw": _own_adamw}[state["case"]["op"]](cce, state)


def run(state):
    return _run_own(state) if own else _run_plain(state)


# -------------------------------------------------------------------- work
def work(case):
    if case["op"] == "adamw":
        n = sum(math.prod(s) for s in _shapes(case))
        each = 2 * BYTES[case["p"]] + BYTES[case["g"]] + (8 if case["master"] else 0) - (BYTES[case["p"]] if case["master"] else 0)
        each += 16 if case["bits"] == 32 else 4 + 16 / BLOCK  # both states and their scales, read and written
        return {"bytes": n * each, "flops": 16 * n}
    m, d, n = _rows(case), case["dim"], case["out"]
    e = BYTES[case["x"]]
    mats = 2 if case["op"] == "gated" else 1
    y = BYTES[case.get("y", case["x"])]
    bias = BYTES[case["bias"]] * n if case.get("bias") else 0
    ahead = 2 * m * d * n * mats
    x, w = m * d * e, n * d * e * mats
    if case["pass"] == "forward":
        return {"bytes": x + w + bias + m * n * y * (2 if case.get("residual") else 1), "flops": ahead}
    # x, the weights and dy in, dx and the parameters' gradients out
    back = 2 * x + 2 * w + bias + m * n * y
    if case["pass"] == "backward":
        kept = m * n * e * mats if case.get("act") != "none" else 0
        return {"bytes": back + kept, "flops": 2 * ahead}
    return {"bytes": back + bias + m * n * y * (2 if case.get("residual") else 1), "flops": 3 * ahead}


# ------------------------------------------------------------ in 64 bits
@torch.no_grad()
def exact(case, seed):
    state = prepare(case, seed)
    if case["op"] == "adamw":
        return _exact_adamw(case, state)
    # fp64 products run at about one TFLOP/s
    if work(case)["flops"] > 1.2e13:
        return None
    d, n, act = case["dim"], case["out"], case["act"]
    x = state["x"].double().reshape(-1, d)
    names = ("wg", "wu") if case["op"] == "gated" else ("w",)
    weights = [state[k].double() for k in names]
    pre = [state["z" + k].double().reshape(-1, n) if case["pass"] == "backward" else torch.einsum("md,nd->mn", x, w)
           for k, w in zip(names, weights)]
    if "b" in state and case["pass"] != "backward":
        pre = [z + state["b"].double() for z in pre]
    a = _exact_activation(act, pre[0])
    out = {}
    if case["pass"] != "backward":
        y = a * pre[1] if case["op"] == "gated" else a
        out["y"] = y + state["r"].double().reshape(-1, n) if "r" in state else y
    if case["pass"] != "forward":
        dy = state["dy"].double().reshape(-1, n)
        slope = _exact_slope(act, pre[0])
        grads = [dy * pre[1] * slope, dy * a] if case["op"] == "gated" else [dy * slope]
        out["dx"] = sum(torch.einsum("mn,nd->md", g, w) for g, w in zip(grads, weights))
        for k, g in zip(names, grads):
            out["d" + k] = torch.einsum("mn,md->nd", g, x)
        if "b" in state:
            out["db"] = torch.einsum("mn->n", grads[0])
    return out


def _exact_activation(act, z):
    if act == "none":
        return z
    if act == "relu":
        return torch.where(z > 0, z, torch.zeros_like(z))
    if act == "gelu":  # z times the normal distribution function
        return z * torch.special.ndtr(z)
    # z times a logistic function: tanh(u) is 2 sigmoid(2 u) - 1
    return z * torch.sigmoid(z if act == "silu" else 2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z.pow(3)))


def _exact_slope(act, z):
    if act == "none":
        return torch.ones_like(z)
    if act == "relu":
        return torch.heaviside(z, torch.zeros_like(z))
    if act == "gelu":
        return torch.special.ndtr(z) + z * torch.exp(-z.pow(2) / 2) / math.sqrt(2 * math.pi)
    u, du = (z, 1.0) if act == "silu" else (2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z.pow(3)),
                                            2 * math.sqrt(2 / math.pi) * (1 + 0.134145 * z.pow(2)))
    s = torch.sigmoid(u)
    return s + z * s * torch.sigmoid(-u) * du


def _exact_adamw(case, state):
    t = case["t"]
    g = state["g"].double()
    if case["clip"]:
        g = g * min(1.0, state["max_norm"] / (float(state["norm"]) + CLIP_EPS))
    if case["bits"] == 32:
        m, v = state["m"].double(), state["v"].double()
    else:
        m = state["m"].double() * state["ms"].double().repeat_interleave(BLOCK)
        v = (state["r"].double() * state["rs"].double().repeat_interleave(BLOCK)).pow(2)
    m = m + (1 - BETA1) * (g - m)
    v = v + (1 - BETA2) * (g.pow(2) - v)
    old = (state["master"] if case["master"] else state["p"]).double()
    new = old - LR * (DECAY * old + (m / (1 - BETA1 ** t)) / ((v / (1 - BETA2 ** t)).sqrt() + EPS))
    out = {"p": new}
    if case["master"]:
        out["master"] = new
    if case["bits"] == 32:
        return out | {"m": m, "v": v}
    # which neighbour a value is rounded to is for the random words to say
    words = _random_words(state, m.numel())
    for k, values, word in (("m", m, words & 0xFFFF), ("r", v.sqrt(), words >> 16)):
        most = values.abs().view(-1, BLOCK).amax(1)
        most = torch.where(most < TINY, 0.0, most)
        a = (values.abs() / most.repeat_interleave(BLOCK) * TOP).nan_to_num(0.0)
        fine = torch.exp2(torch.floor(torch.log2(a.clamp(min=2.0 ** -6))) - 3)
        low = torch.floor(a / fine) * fine
        up = (a - low) / fine + word.double() / 65536 >= 1
        q = torch.where(up, low + fine, low).clamp(max=TOP)
        if k == "r":
            q = torch.where(values > 0, q.clamp(min=2.0 ** -9), q)
        out[k], out[k + "s"] = q * values.sign(), most / TOP
    return out
