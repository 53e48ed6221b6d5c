"""Cases of the operators around the loss head: layer norm, RMS norm, the
global gradient norm and gradient clipping.

The classifier head reads hidden states that a norm has just produced, and a
training step clips the gradients that its backward pass leaves before the
optimiser reads them.  Each case is one call (or one forward and backward) of
such an operator, in its plain form (elementary torch operations in 32 bits)
or, with `own` set, through linear_cross_entropy_gb300.
"""
import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
BYTES = {"bf16": 2, "fp16": 2, "fp32": 4}
CLIP_EPS = 1e-6  # added to the norm before the division, as torch's clipping does


# ------------------------------------------------------------------- cases
def _rows_case(name, op, pass_, batch, seq, dim, x="bf16", y=None, w=None, offset=0.0, shift=False):
    return {"name": name, "op": op, "pass": pass_, "batch": batch, "seq": seq, "dim": dim, "x": x,
            "y": y or x, "w": w or x, "offset": offset, "shift": shift}


def _grads_case(name, op, layers, dim, vocab, g="bf16", out="fp32", norm="2", bucket=False, fraction=0.3):
    return {"name": name, "op": op, "layers": layers, "dim": dim, "vocab": vocab, "g": g, "out": out, "norm": norm,
            "bucket": bucket, "fraction": fraction}


def listed():
    return [
        # decoding one token: the last norm before the logits, all latency
        _rows_case("layer norm 1 token", "layer_norm", "forward", 1, 1, 896),
        # decoding a small odd batch, half precision
        _rows_case("rms norm 33 tokens", "rms_norm", "forward", 33, 1, 4096, x="fp16"),
        # the forward of a Gemma-2-2B-shaped batch
        _rows_case("layer norm forward", "layer_norm", "forward", 4, 2048, 2304),
        # per-head normalisation of the queries of 4,096 tokens with 16 heads
        _rows_case("rms norm heads", "rms_norm", "forward", 4096, 16, 128),
        # the backward of a Qwen2.5-0.5B-shaped batch, 32-bit parameters
        _rows_case("layer norm backward", "layer_norm", "backward", 1, 4096, 896, w="fp32"),
        # the backward of a Gemma-2-2B-shaped batch, whose weights are stored minus one
        _rows_case("rms norm backward", "rms_norm", "backward", 4, 2048, 2304, offset=1.0),
        # 32-bit residual stream normalised to the 16-bit hidden states of a Llama-3-8B-shaped head
        _rows_case("layer norm step mixed", "layer_norm", "step", 8, 2048, 4096, x="fp32", y="bf16"),
        # every token but the last of each sequence predicts the next one; odd width
        _rows_case("layer norm step odd", "layer_norm", "step", 7, 147, 1001, x="fp16", shift=True),
        # training on the long-context batch of 65,536 tokens
        _rows_case("rms norm step long", "rms_norm", "step", 1, 65536, 2048),
        # the head alone being trained at its smallest size
        _grads_case("clip tiny head", "clip", 0, 128, 4096, out="bf16"),
        # gradient norm of a Qwen2.5-0.5B-shaped head, for logging
        _grads_case("grad norm head", "grad_norm", 0, 896, 151936),
        # a whole 24-layer model: 16-bit gradients clipped into the optimiser's 32-bit buffer
        _grads_case("clip model", "clip", 24, 896, 151936),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def _width(rng, lo, hi):
    """An odd multiple of 1, 8, 128 or 512."""
    step = rng.choice((1, 8, 128, 512))
    return step * (_log(rng, max(1, lo // step), max(1, (hi - step) // step)) | 1)


def draw(rng):
    case = _drawn(rng)
    del case["name"]
    return case


def _drawn(rng):
    if rng.random() < 0.3:
        dim = _width(rng, 64, 1024)
        layers = rng.choice((0, 0, _log(rng, 1, 24)))
        g = rng.choice(("bf16", "bf16", "fp16", "fp32"))
        return _grads_case("", rng.choice(("grad_norm", "clip", "clip")), layers, dim, _log(rng, 1000, 131072), g=g,
                           out=rng.choice((g, "fp32")), norm=rng.choice(("2", "2", "2", "inf")),
                           bucket=rng.random() < 0.3, fraction=rng.choice((0.01, 0.3, 2.0)))
    dim = _width(rng, 64, 16384)
    rows = _log(rng, 1, min(65536, 65536 * 2048 // dim))
    batch = min(rows, rng.choice((1, 2, 7, 16)))
    seq = max(1, rows // batch)
    x, y = rng.choice((("bf16", "bf16"), ("bf16", "bf16"), ("fp16", "fp16"), ("fp32", "fp32"), ("fp32", "bf16")))
    op = rng.choice(("layer_norm", "rms_norm"))
    return _rows_case("", op, rng.choice(("forward", "backward", "step")), batch, seq, dim, x=x, y=y,
                      w=rng.choice((x, "fp32")), offset=rng.choice((0.0, 1.0)) if op == "rms_norm" else 0.0,
                      shift=seq > 1 and rng.random() < 0.25)


def _rows(case):
    return case["batch"] * (case["seq"] - 1 if case["shift"] else case["seq"])


def _shapes(case):
    """The parameters of a decoder of that width (attention, gated MLP, norms) and of its head."""
    d = case["dim"]
    layer = [(d, d)] * 4 + [(d,)] * 3 + [(4 * d, d)] * 2 + [(d, 4 * d)] + [(d,)] * 2
    return layer * case["layers"] + [(d,), (d,), (case["vocab"], d)]


def _eps(case):
    return 1e-5 if case["op"] == "layer_norm" else 1e-6


# ------------------------------------------------------------------ inputs
def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def randn(*shape):
        return torch.randn(shape, generator=gen, device="cuda")

    if case["op"] in ("clip", "grad_norm"):
        return _prepare_grads(case, gen, randn)
    b, s, d = case["batch"], case["seq"], case["dim"]
    # hidden states: a mean, channels of unequal size and a few that stand out
    scale = torch.exp(0.3 * randn(d))
    scale[::97] *= 8.0
    x = (randn(b, s, d) * scale + 0.2 * randn(d)).to(TYPES[case["x"]])
    x = x[:, :-1] if case["shift"] else x
    state = {"case": case, "x": x, "w": (1.0 - case["offset"] + 0.1 * randn(d)).to(TYPES[case["w"]])}
    if case["op"] == "layer_norm":
        state["b"] = (0.1 * randn(d)).to(TYPES[case["w"]])
    if case["pass"] != "forward":
        dy = (1e-2 * randn(b, s, d)).to(TYPES[case["y"]])
        state["dy"] = dy[:, :-1] if case["shift"] else dy
    if case["pass"] == "backward":  # what the forward pass left
        mean, rstd = _statistics(case, x.float())
        if mean is not None:
            state["mean"] = mean.reshape(-1)
        state["rstd"] = rstd.reshape(-1)
    if case["pass"] == "step":
        for k in ("x", "w", "b"):
            if k in state:
                state[k].requires_grad_()
    return state


def _prepare_grads(case, gen, randn):
    shapes = _shapes(case)
    sizes = [math.prod(s) for s in shapes]
    # each tensor's gradient has a scale of its own; rows of rare tokens get none
    scales = torch.exp(randn(len(shapes)) - 6.0)
    grads = [randn(*s) * scales[i] for i, s in enumerate(shapes)]
    rare = torch.rand((shapes[-1][0], 1), generator=gen, device="cuda") < 0.1
    grads[-1] = grads[-1].masked_fill(rare, 0.0)
    total = float(torch.stack([g.square().sum() for g in grads]).sum().sqrt())
    grads = [g.to(TYPES[case["g"]]) for g in grads]
    if case["bucket"]:  # gradients that live in one flat bucket
        flat = torch.cat([g.reshape(-1) for g in grads])
        grads = [v.view(s) for v, s in zip(flat.split(sizes), shapes)]
    if case["norm"] == "inf":
        total = float(torch.stack([g.abs().max().float() for g in grads]).max())
    state = {"case": case, "grads": grads}
    if case["op"] == "clip":
        state["max_norm"] = case["fraction"] * total
        state["flat"] = torch.empty(sum(sizes), dtype=TYPES[case["out"]], device="cuda")
        state["outs"] = [v.view(s) for v, s in zip(state["flat"].split(sizes), shapes)]
    return state


# -------------------------------------------------------------- plain forms
def _statistics(case, x):
    if case["op"] == "layer_norm":
        mean = x.mean(-1, keepdim=True)
        return mean, torch.rsqrt((x - mean).square().mean(-1, keepdim=True) + _eps(case))
    return None, torch.rsqrt(x.square().mean(-1, keepdim=True) + _eps(case))


def _plain_forward(case, x, w, b, mean, rstd):
    xhat = (x - mean) * rstd if mean is not None else x * rstd
    y = xhat * (w.float() + case["offset"])
    return (y + b.float() if b is not None else y).to(TYPES[case["y"]])


def _plain_backward(case, x, w, dy, mean, rstd):
    xhat = (x - mean) * rstd if mean is not None else x * rstd
    dy = dy.float()
    g = dy * (w.float() + case["offset"])
    dx = g - xhat * (g * xhat).mean(-1, keepdim=True)
    if mean is not None:
        dx = dx - g.mean(-1, keepdim=True)
    d = case["dim"]
    out = {"dx": (dx * rstd).to(TYPES[case["x"]]), "dw": (dy * xhat).reshape(-1, d).sum(0).to(w.dtype)}
    if mean is not None:
        out["db"] = dy.reshape(-1, d).sum(0).to(w.dtype)
    return out


def _plain_norm(case, grads):
    if case["norm"] == "inf":
        return torch.stack([g.abs().max().float() for g in grads]).max()
    return torch.stack([g.float().square().sum() for g in grads]).sum().sqrt()


@torch.no_grad()
def _run_plain(state):
    case = state["case"]
    if case["op"] in ("clip", "grad_norm"):
        norm = _plain_norm(case, state["grads"])
        if case["op"] == "grad_norm":
            return norm
        coef = (state["max_norm"] / (norm + CLIP_EPS)).clamp(max=1.0)
        clipped = torch.cat([(g.float() * coef).to(TYPES[case["out"]]).reshape(-1) for g in state["grads"]])
        return {"norm": norm, "clipped": clipped}
    x = state["x"].float()
    if case["pass"] == "backward":
        rstd = state["rstd"].view(*x.shape[:-1], 1)
        mean = state["mean"].view(*x.shape[:-1], 1) if "mean" in state else None
        return _plain_backward(case, x, state["w"], state["dy"], mean, rstd)
    mean, rstd = _statistics(case, x)
    out = {"y": _plain_forward(case, x, state["w"], state.get("b"), mean, rstd)}
    if case["pass"] == "step":
        out |= _plain_backward(case, x, state["w"], state["dy"], mean, rstd)
    return out


# ----------------------------------------------------------- the operators
def _forward_own(cce, case, state):
    if case["op"] == "layer_norm":
        return cce.layer_norm(state["x"], state["w"], state["b"], eps=_eps(case), out_dtype=TYPES[case["y"]])
    return cce.rms_norm(state["x"], state["w"], eps=_eps(case), weight_offset=case["offset"],
                        out_dtype=TYPES[case["y"]])


def _run_own(state):
    import linear_cross_entropy_gb300 as cce

    case = state["case"]
    if case["op"] == "grad_norm":
        return cce.cce_grad_norm(state["grads"], norm_type=float(case["norm"]))
    if case["op"] == "clip":
        norm = cce.cce_clip_grads(state["grads"], state["max_norm"], norm_type=float(case["norm"]), out=state["outs"])
        return {"norm": norm, "clipped": state["flat"]}
    if case["pass"] == "forward":
        return {"y": _forward_own(cce, case, state)}
    if case["pass"] == "backward":
        if case["op"] == "layer_norm":
            grads = cce.cce_layer_norm_backward(state["dy"], state["x"], state["w"], state["mean"], state["rstd"])
        else:
            grads = cce.cce_rms_norm_backward(state["dy"], state["x"], state["w"], state["rstd"],
                                              weight_offset=case["offset"])
        return dict(zip(("dx", "dw", "db"), grads))
    y = _forward_own(cce, case, state)
    inputs = [state[k] for k in ("x", "w", "b") if k in state]
    return {"y": y.detach()} | dict(zip(("dx", "dw", "db"), torch.autograd.grad(y, inputs, state["dy"])))


def run(state):
    return _run_own(state) if own else _run_plain(state)


# -------------------------------------------------------------------- work
def work(case):
    if case["op"] in ("clip", "grad_norm"):
        n = sum(math.prod(s) for s in _shapes(case))
        if case["op"] == "grad_norm":
            return {"bytes": n * BYTES[case["g"]] + 4, "flops": 2 * n}
        return {"bytes": n * (BYTES[case["g"]] + BYTES[case["out"]]) + 4, "flops": 3 * n}
    n, d = _rows(case), case["dim"]
    x, y, w = BYTES[case["x"]], BYTES[case["y"]], BYTES[case["w"]]
    layer = case["op"] == "layer_norm"
    params = (2 if layer else 1) * d * w
    forward, backward = (8 if layer else 4) * n * d, (14 if layer else 11) * n * d
    if case["pass"] == "forward":
        return {"bytes": n * d * (x + y) + params, "flops": forward}
    if case["pass"] == "backward":  # x, dy and the statistics in, dx and the parameters' gradients out
        return {"bytes": n * d * (2 * x + y) + n * (8 if layer else 4) + d * w + params, "flops": backward}
    return {"bytes": n * d * (2 * x + 2 * y) + 2 * params, "flops": forward + backward}


# ------------------------------------------------------------ in 64 bits
@torch.no_grad()
def exact(case, seed):
    state = prepare(case, seed)
    if case["op"] in ("clip", "grad_norm"):
        return _exact_grads(case, state)
    d = case["dim"]
    x = state["x"].double().reshape(-1, d)
    gain = state["w"].double() + case["offset"]
    if case["pass"] == "backward":
        centre = state["mean"].double().unsqueeze(1) if "mean" in state else 0.0
        inv = state["rstd"].double().unsqueeze(1)
    else:
        centre = x.sum(1, keepdim=True) / d if case["op"] == "layer_norm" else 0.0
        inv = 1.0 / ((x - centre).pow(2).sum(1, keepdim=True) / d + _eps(case)).sqrt()
    z = (x - centre) * inv
    out = {}
    if case["pass"] != "backward":
        out["y"] = z * gain + (state["b"].double() if "b" in state else 0.0)
    if case["pass"] != "forward":
        dy = state["dy"].double().reshape(-1, d)
        dz = dy * gain
        along = torch.einsum("nd,nd->n", dz, z).unsqueeze(1)
        total = dz.sum(1, keepdim=True) if case["op"] == "layer_norm" else 0.0
        out["dx"] = (d * dz - total - z * along) * (inv / d)
        out["dw"] = torch.einsum("nd,nd->d", dy, z)
        if case["op"] == "layer_norm":
            out["db"] = dy.sum(0)
    return out


def _exact_grads(case, state):
    flat = torch.cat([g.double().reshape(-1) for g in state["grads"]])
    norm = flat.abs().max() if case["norm"] == "inf" else torch.linalg.vector_norm(flat)
    if case["op"] == "grad_norm":
        return norm
    return {"norm": norm, "clipped": flat * min(1.0, state["max_norm"] / (float(norm) + CLIP_EPS))}
