"""Host side of AdamW without a GPU: refusals of the C ABI before any launch, of
the binding and of the optimiser."""
import ctypes
import math
import os
import re

import pytest
import torch
import torch.autograd.forward_ad as fwAD
from torch.fx.experimental.proxy_tensor import make_fx

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 1 << 20  # an aligned non-null host integer: never dereferenced, checks fail first
MiB = 1 << 20
F32, F16, BF16 = 0, 1, 2


@pytest.fixture(scope="module")
def lib():
    from tests.conftest import build_library
    build_library()
    from linear_cross_entropy_gb300 import _lib
    return _lib.load()


@pytest.fixture(scope="module")
def cce(lib):
    import linear_cross_entropy_gb300
    return linear_cross_entropy_gb300


def _tensor(**kw):
    from linear_cross_entropy_gb300._lib import AdamWTensor
    a = dict(grad=1 * MiB, param=2 * MiB, master=0, exp_avg=3 * MiB, exp_avg_sq=4 * MiB, exp_avg_scale=5 * MiB,
             rms_scale=6 * MiB, n=1000, grad_type=BF16, param_type=BF16, weight_decay=0.1)
    assert kw.keys() <= a.keys()
    return AdamWTensor(*(a | kw).values())


def _step(lib, tensors=None, bits=32, count=None, options=True, **kw):
    from linear_cross_entropy_gb300._lib import AdamWOptions, AdamWTensor
    tensors = [_tensor()] if tensors is None else tensors
    table = (AdamWTensor * max(1, len(tensors)))(*tensors)
    a = dict(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, step=1, step_ptr=0, lr_ptr=0, norm=0, max_norm=1.0, eps_norm=1e-6,
             seed=0)
    assert kw.keys() <= a.keys()
    o = ctypes.byref(AdamWOptions(*(a | kw).values())) if options else None
    return lib.cce_adamw_step(table if tensors is not None else None, len(tensors) if count is None else count, bits, o, 0)


def test_declared_symbols(lib):
    src = open(os.path.join(ROOT, "include", "cce_optim.h")).read()
    names = set(re.findall(r"^(?:int|cce_status) (cce_[a-z0-9_]+)\s*\(", src, flags=re.M))
    assert names == {"cce_optim_abi_version", "cce_adamw_step"} and all(hasattr(lib, n) for n in names)
    assert lib.cce_optim_abi_version() == 100


@pytest.mark.parametrize("kw,status", [
    (dict(bits=16), 4), (dict(beta1=1.0), 4), (dict(beta1=-0.1), 4), (dict(beta2=1.5), 4), (dict(beta2=math.nan), 4),
    (dict(lr=-1.0), 4), (dict(lr=math.inf), 4), (dict(eps=math.nan), 4), (dict(eps=-1.0), 4), (dict(step=0), 4),
    (dict(norm=FAKE, max_norm=-1.0), 4), (dict(norm=FAKE, max_norm=math.nan), 4), (dict(norm=FAKE, eps_norm=-1.0), 4),
    (dict(norm=FAKE + 2), 3), (dict(step_ptr=FAKE + 4), 3), (dict(lr_ptr=FAKE + 1), 3), (dict(count=-1), 2),
    (dict(options=False), 1),
])
def test_options_are_checked(lib, kw, status):
    assert _step(lib, **kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(grad=0), 1), (dict(param=0), 1), (dict(exp_avg=0), 1), (dict(exp_avg_sq=0), 1), (dict(n=-1), 2),
    (dict(n=1 << 35), 2), (dict(grad_type=3), 4), (dict(param_type=-1), 4), (dict(weight_decay=-1.0), 4),
    (dict(weight_decay=math.nan), 4), (dict(grad=MiB + 1), 3), (dict(param=MiB + 1), 3), (dict(master=MiB + 2), 3),
    (dict(param=1 * MiB), 4), (dict(param=1 * MiB + 1998), 4), (dict(exp_avg=4 * MiB), 4), (dict(master=2 * MiB), 4),
])
def test_tensors_are_checked(lib, kw, status):
    for bits in (8, 32):
        assert _step(lib, [_tensor(**kw)], bits) == status
        assert _step(lib, [_tensor(param=64 * MiB, exp_avg=65 * MiB, exp_avg_sq=66 * MiB, exp_avg_scale=67 * MiB,
                                   rms_scale=68 * MiB), _tensor(**kw)], bits) == status


def test_each_kind_of_state_is_checked(lib):
    for kw in (dict(exp_avg=3 * MiB + 2), dict(exp_avg_sq=4 * MiB + 1)):
        assert _step(lib, [_tensor(**kw)], 32) == 3
    for kw, status in ((dict(exp_avg_scale=0), 1), (dict(rms_scale=0), 1), (dict(rms_scale=FAKE + 2), 3),
                       (dict(rms_scale=5 * MiB + 12), 4), (dict(exp_avg_scale=3 * MiB + 996), 4)):
        assert _step(lib, [_tensor(**kw)], 8) == status
    assert _step(lib, [_tensor(), _tensor()]) == 4  # the same tensor twice


@pytest.mark.skipif(torch.cuda.is_available(), reason="would launch on fake pointers when a GPU is present")
def test_valid_arguments_without_gpu_report_cuda_error(lib):
    for bits in (8, 32):
        assert _step(lib, bits=bits) in (6, 7)
        assert _step(lib, [], bits) in (6, 7)
        assert _step(lib, [_tensor(grad=0, n=0)], bits) in (6, 7)
        assert _step(lib, [_tensor(master=16 * MiB)], bits, norm=FAKE, max_norm=math.inf) in (6, 7)
    # two tensors may share a gradient; states of 8 bits start anywhere, 32-bit states read no scales
    other = dict(param=12 * MiB, exp_avg=13 * MiB, exp_avg_sq=14 * MiB, exp_avg_scale=15 * MiB, rms_scale=16 * MiB)
    assert _step(lib, [_tensor(), _tensor(**other)]) in (6, 7)
    assert _step(lib, [_tensor(exp_avg=3 * MiB + 1)], 8) in (6, 7)
    assert _step(lib, [_tensor(exp_avg_scale=0, rms_scale=1)], 32) in (6, 7)
    assert _step(lib, step=0, step_ptr=FAKE) in (6, 7)


def test_binding_refuses(cce):
    t = [torch.zeros(4)]
    with pytest.raises(ValueError, match="CUDA"):
        cce.cce_adamw_step(t, t, t, t, 1, lr=0.1)
    with pytest.raises(ValueError, match="CUDA"):
        cce.cce_adamw8_step(t, t, t, t, t, t, 1, lr=0.1)
    for call, match in ((lambda: cce.cce_adamw_step(t, [], t, t, 1, lr=0.1), "grads"),
                        (lambda: cce.cce_adamw_step(t, t, t, [], 1, lr=0.1), "states"),
                        (lambda: cce.cce_adamw8_step(t, t, t, [], t, t, 1, lr=0.1), "states"),
                        (lambda: cce.cce_adamw_step(t, t, t, t, 0, lr=0.1), "step"),
                        (lambda: cce.cce_adamw_step(t, t, t, t, 1, lr=0.1, max_norm=1.0), "together"),
                        (lambda: cce.cce_adamw_step(t, t, t, t, 1, lr=0.1, weight_decay=[]), "weight_decay")):
        with pytest.raises(ValueError, match=match):
            call()
    cce.cce_adamw_step([], [], [], [], 1, lr=0.1)
    cce.cce_adamw8_step([], [], [], [], [], [], 1, lr=0.1)
    assert cce.adamw_scales(0) == 0 and cce.adamw_scales(256) == 1 and cce.adamw_scales(257) == 2


def test_tangents_and_tracing_are_refused(cce):
    t = torch.zeros(4)
    with fwAD.dual_level():
        d = fwAD.make_dual(torch.zeros(4), torch.ones(4))
        for p, g in ((d, t), (t, d)):
            with pytest.raises(NotImplementedError, match="tangent"):
                cce.cce_adamw_step([p], [g], [t], [t], 1, lr=0.1)

    def call(x):
        cce.cce_adamw_step([x], [t], [t], [t], 1, lr=0.1)
        return x
    with pytest.raises(NotImplementedError, match="traced"):
        torch.jit.trace(call, (t,))
    with pytest.raises(NotImplementedError, match="traced"):
        make_fx(call)(t)


def test_optimiser_refuses(cce):
    p = [torch.nn.Parameter(torch.zeros(4))]
    for kw in (dict(state_bits=16), dict(lr=-1.0), dict(lr=math.nan), dict(betas=(0.9, 1.0)), dict(eps=-1.0),
               dict(weight_decay=-0.1)):
        with pytest.raises(ValueError):
            cce.AdamW(p, **kw)
    opt = cce.AdamW(p)
    opt.step()  # nothing has a gradient
    p[0].grad = torch.zeros(4)
    with pytest.raises(ValueError, match="CUDA"):
        opt.step()
