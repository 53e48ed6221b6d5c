"""AdamW over many tensors in one launch, with states in 32 or in 8 bits.

    opt = AdamW(model.parameters(), lr=1e-3, state_bits=8)
    loss.backward()
    norm = cce_grad_norm([p.grad for p in model.parameters()])
    opt.step(grad_norm=norm, max_norm=1.0)      # clips on the way: no pass of its own
    opt.zero_grad()

cce_adamw_step and cce_adamw8_step are the direct calls on lists of tensors.
With g the gradient times min(1, max_norm / (grad_norm + 1e-6)):

    m = beta1 m + (1 - beta1) g,  v = beta2 v + (1 - beta2) g^2
    w = w (1 - lr weight_decay) - lr / (1 - beta1^t) m / (sqrt(v / (1 - beta2^t)) + eps)

in fp32, for parameters and gradients of bf16, fp16 or fp32.  With fp32 masters,
w is the master and the parameter is w rounded to its type.  In 8 bits a block of
256 values of m, or of the root of v, is float8_e4m3fn values and an fp32 scale,
rounded at random with numbers that (seed, step, place) fix, so that averages move
although a step's change is below a rounding; a NaN or infinity in a gradient makes
the states of its block NaN.

Parameters, masters and states are written in place; they must be dense and not
overlap.  Calls run on the current stream of the parameters' device and can be
captured into a CUDA graph, with step (and lr, where it changes) as device tensors.
Arguments that do not fit raise ValueError, a status of the library CCEError;
forward-mode derivatives and tracing NotImplementedError.
"""
from __future__ import annotations

import torch

from . import _native
from .grads import CLIP_EPS

BLOCK = 256  # values that share a scale in 8-bit states


def adamw_scales(numel) -> int:
    """How many scales each 8-bit state of a tensor with that many values has."""
    return -(-numel // BLOCK)


def _tensor_or_none(value):
    """A device tensor in place of a number."""
    return value if type(value) not in (int, float) and isinstance(value, torch.Tensor) else None


def _step(params, grads, states, bits, step, lr, betas, eps, weight_decay, masters, grad_norm, max_norm, seed, stream):
    params = list(params)
    n = len(params)
    args = [params]
    names = ("grads", "masters", "states", "states", "states", "states")
    for name, given in zip(names, (grads, (None,) * n if masters is None else masters, *states)):
        given = list(given)
        if len(given) != n:
            raise ValueError(f"{name} must have one tensor for each of the {n} params, got {len(given)}")
        args.append(given)
    if type(weight_decay) is float or isinstance(weight_decay, (int, float)):
        decay = [float(weight_decay)]
    else:
        decay = [float(d) for d in weight_decay]
        if len(decay) != n:
            raise ValueError(f"weight_decay must be a number or one for each of the {n} params, got {len(decay)}")
    if (grad_norm is None) != (max_norm is None):
        raise ValueError("grad_norm and max_norm come together")
    max_norm = 0.0 if max_norm is None else float(max_norm)
    if not max_norm >= 0.0:
        raise ValueError(f"max_norm must be at least 0, got {max_norm}")
    at, lr_at = _tensor_or_none(step), _tensor_or_none(lr)
    step = 1 if at is not None else int(step)
    if step < 1:
        raise ValueError(f"step must be at least 1, got {step}")
    if not params:
        return
    if bits == 32:
        args += [], []
    beta1, beta2 = betas
    args += (bits, step, at, 0.0 if lr_at is not None else float(lr), lr_at, float(beta1), float(beta2), float(eps), decay,
             grad_norm, max_norm, CLIP_EPS, int(seed) & 0xFFFFFFFF)
    if stream is None:
        _native.adamw_step(*args)
    else:
        with torch.cuda.stream(stream):
            _native.adamw_step(*args)


def cce_adamw_step(params, grads, exp_avgs, exp_avg_sqs, step, *, lr, betas=(0.9, 0.999), eps=1e-8, weight_decay=0.01,
                   masters=None, grad_norm=None, max_norm=None, stream=None):
    """One AdamW update in place: params, exp_avgs (m), exp_avg_sqs (v) and the
    masters, lists of tensors.  m, v and masters are float32.

    step: the number of this update, from 1 on, or a device tensor (int64) that
    holds it; lr: a number or a device tensor (float32); weight_decay: a number or
    one for each tensor; masters: None, or a tensor or None for each.  With grad_norm
    (a device tensor, float32) and max_norm the gradients count clipped; a NaN norm
    makes the update NaN."""
    _step(params, grads, (exp_avgs, exp_avg_sqs), 32, step, lr, betas, eps, weight_decay, masters, grad_norm, max_norm,
          0, stream)


def cce_adamw8_step(params, grads, exp_avgs, exp_avg_scales, exp_avg_rms, rms_scales, step, *, lr, betas=(0.9, 0.999),
                    eps=1e-8, weight_decay=0.01, masters=None, grad_norm=None, max_norm=None, seed=0, stream=None):
    """The same with states in 8 bits: m is exp_avgs times its block's scale,
    sqrt(v) exp_avg_rms times its own; float8_e4m3fn tensors of the parameters'
    shapes and strides, and float32 scales [adamw_scales(numel)], one for each 256
    values in memory order.  All zeros are the states to begin with."""
    _step(params, grads, (exp_avgs, exp_avg_rms, exp_avg_scales, rms_scales), 8, step, lr, betas, eps, weight_decay,
          masters, grad_norm, max_norm, seed, stream)


class AdamW(torch.optim.Optimizer):
    """AdamW on cce_adamw_step and cce_adamw8_step, one launch for each kind of
    tensor.

    state_bits: 32, or 8 for tensors of at least min_8bit_size values (others keep
    32).  master_weights: 16-bit parameters get an fp32 master, made from them at
    their first step.  seed: of the 8-bit states' rounding.  capturable: steps are
    counted on the device, one count for a group, so that step() can be captured into
    a CUDA graph (after one step outside of the capture, which makes the states); lr
    may be a device tensor."""

    def __init__(self, params, lr=1e-3, betas=(0.9, 0.999), eps=1e-8, weight_decay=0.01, *, state_bits=32,
                 master_weights=False, min_8bit_size=4096, seed=0, capturable=False):
        super().__init__(params, dict(lr=lr, betas=betas, eps=eps, weight_decay=weight_decay, state_bits=state_bits,
                                      master_weights=master_weights, min_8bit_size=min_8bit_size, seed=seed,
                                      capturable=capturable))

    def add_param_group(self, param_group):
        """As of any optimiser; a group's own options are checked as the optimiser's are."""
        options = self.defaults | param_group
        state_bits, lr, betas = options["state_bits"], options["lr"], options["betas"]
        eps, weight_decay = options["eps"], options["weight_decay"]
        if state_bits not in (8, 32):
            raise ValueError(f"state_bits must be 8 or 32, got {state_bits}")
        if not isinstance(lr, torch.Tensor) and not lr >= 0.0:
            raise ValueError(f"lr must be at least 0, got {lr}")
        if not all(0.0 <= b < 1.0 for b in betas):
            raise ValueError(f"betas must be in [0, 1), got {betas}")
        if not eps >= 0.0 or not weight_decay >= 0.0:
            raise ValueError(f"eps and weight_decay must be at least 0, got {eps} and {weight_decay}")
        super().add_param_group(param_group)

    def _counter(self, device, group):
        """The group's count of steps on that device."""
        for q in group["params"]:
            if q.device == device and "step" in self.state.get(q, {}):
                return self.state[q]["step"]
        return torch.zeros((), dtype=torch.int64, device=device)

    def _state_of(self, p, group):
        state = self.state[p]
        if not state:
            state["step"] = self._counter(p.device, group) if group["capturable"] else 0

            def zeros(dtype):
                return torch.zeros_like(p, dtype=dtype, requires_grad=False, memory_format=torch.preserve_format)

            if group["state_bits"] == 8 and p.numel() >= group["min_8bit_size"]:
                state["exp_avg"], state["exp_avg_rms"] = (zeros(torch.uint8).view(torch.float8_e4m3fn) for _ in "mr")
                for k in ("exp_avg_scale", "rms_scale"):
                    state[k] = torch.zeros(adamw_scales(p.numel()), dtype=torch.float32, device=p.device)
            else:
                state["exp_avg"], state["exp_avg_sq"] = zeros(torch.float32), zeros(torch.float32)
            if group["master_weights"] and p.dtype != torch.float32:
                state["master"] = p.detach().float()
        return state

    @torch.no_grad()
    def step(self, closure=None, *, grad_norm=None, max_norm=None):
        """One update of the parameters that have a gradient.  grad_norm and
        max_norm as in cce_adamw_step."""
        loss = None
        if closure is not None:
            with torch.enable_grad():
                loss = closure()
        for index, group in enumerate(self.param_groups):
            calls = {}  # parameters that step together: one device, one number of steps, one kind of state
            counted = set()
            for p in group["params"]:
                if p.grad is None:
                    continue
                state = self._state_of(p, group)
                if isinstance(state["step"], torch.Tensor):
                    if id(state["step"]) not in counted:
                        state["step"].add_(1)
                        counted.add(id(state["step"]))
                    when = id(state["step"])
                else:
                    state["step"] += 1
                    when = state["step"]
                calls.setdefault((p.device, when, "rms_scale" in state), []).append((p, state))
            for (_, _, eight), members in calls.items():
                params = [p for p, _ in members]
                states = [s for _, s in members]

                def all_of(key):
                    return [s[key] for s in states]

                more = dict(lr=group["lr"], betas=group["betas"], eps=group["eps"], weight_decay=group["weight_decay"],
                            masters=[s.get("master") for s in states], grad_norm=grad_norm, max_norm=max_norm)
                grads, when = [p.grad for p in params], states[0]["step"]
                if eight:
                    cce_adamw8_step(params, grads, all_of("exp_avg"), all_of("exp_avg_scale"), all_of("exp_avg_rms"),
                                    all_of("rms_scale"), when, seed=group["seed"] + index, **more)
                else:
                    cce_adamw_step(params, grads, all_of("exp_avg"), all_of("exp_avg_sq"), when, **more)
        return loss

    def load_state_dict(self, state_dict):
        """As of any optimiser, but the states keep their own types.  32-bit states and
        masters take the parameters' strides; 8-bit ones, whose scales go by the order
        in memory, are for parameters of the strides that they were made for."""
        super().load_state_dict(state_dict)
        saved = [i for g in state_dict["param_groups"] for i in g["params"]]
        own = [p for g in self.param_groups for p in g["params"]]
        for i, p in zip(saved, own):
            for k, v in state_dict["state"].get(i, {}).items():
                if not isinstance(v, torch.Tensor):
                    continue
                if k in ("exp_avg", "exp_avg_sq", "master") and v.dtype == torch.float32 and v.shape == p.shape:
                    own_order = torch.empty_like(p, dtype=v.dtype, requires_grad=False, memory_format=torch.preserve_format)
                    self.state[p][k] = own_order.copy_(v.detach())
                else:
                    self.state[p][k] = v.detach().to(p.device).clone(memory_format=torch.preserve_format)
        for group in self.param_groups:
            if group["capturable"]:
                shared = {}
                for p in group["params"]:
                    if "step" in self.state.get(p, {}):
                        step = torch.as_tensor(self.state[p]["step"], dtype=torch.int64, device=p.device)
                        self.state[p]["step"] = shared.setdefault(p.device, step)
