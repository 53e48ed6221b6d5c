"""Layer norm and RMS norm: the norm that produces the classifier head's
hidden states, forward and backward, on the library's CUDA kernels.

    y = layer_norm(x, weight, bias)          # last dimension; differentiable
    y = rms_norm(x, weight, weight_offset=1.0)
    loss = linear_cross_entropy(y, C, targets)

x is bf16, fp16 or fp32 with any number of leading dimensions; the result has
x's type, or with out_dtype a 16-bit type from fp32 rows.  Arithmetic and the
saved statistics are fp32.  Rows may be strided (hidden[:, :-1] is read in
place); the result is contiguous.  Calls run on the current stream of x's
device and can be captured into a CUDA graph.
"""
from __future__ import annotations

import torch
from torch.autograd.function import once_differentiable

from . import _lib

TYPES = {torch.float32: 0, torch.float16: 1, torch.bfloat16: 2}
_raw_stream, _current_device = torch._C._cuda_getCurrentRawStream, torch._C._cuda_getDevice

_l = _lib.load()
_layer_forward, _layer_backward = _l.cce_layer_norm_forward, _l.cce_layer_norm_backward
_rms_forward, _rms_backward = _l.cce_rms_norm_forward, _l.cce_rms_norm_backward
_workspace_bytes = _l.cce_norm_backward_workspace_bytes


def norm_backward_workspace_bytes(N, D) -> int:
    return int(_workspace_bytes(N, D))


def _rows(t):
    """(t, inner, row_stride, outer_stride): how the rows of t lie.  Rows that
    are not at one pitch, or in runs at one pitch, or whose elements are apart
    are copied."""
    if t.is_contiguous():
        return t, 1 << 31, t.shape[-1], 0
    shape, stride = t.shape, t.stride()
    runs = []  # (size, stride) of the leading dimensions, outermost first, merged where they continue each other
    if shape[-1] == 1 or stride[-1] == 1:
        for n, s in zip(shape[:-1], stride[:-1]):
            if n == 1:
                continue
            if runs and runs[-1][1] == n * s:
                runs[-1] = (runs[-1][0] * n, s)
            else:
                runs.append((n, s))
        if len(runs) <= 1:
            return t, 1 << 31, runs[0][1] if runs else shape[-1], 0
        if len(runs) == 2:
            return t, runs[1][0], runs[1][1], runs[0][1]
    return t.contiguous(), 1 << 31, shape[-1], 0


def _check(x, weight, bias, name="x"):
    """(N, D, parameter type) of a norm over x's last dimension."""
    if not x.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor (no CPU path)")
    if x.dtype not in TYPES:
        raise ValueError(f"{name} must be bfloat16, float16 or float32, got {x.dtype}")
    index = x.get_device()
    shape = x.shape
    if not shape or shape[-1] < 1:
        raise ValueError(f"{name} needs a last dimension of at least one element, got shape {tuple(shape)}")
    D = shape[-1]
    p_type = None
    for what, p in (("weight", weight), ("bias", bias)):
        if p is None:
            continue
        if p.get_device() != index:
            raise ValueError(f"{what} must be on {x.device}, got {p.device}")
        if p.dtype not in TYPES:
            raise ValueError(f"{what} must be bfloat16, float16 or float32, got {p.dtype}")
        if p.shape != (D,) or not p.is_contiguous():
            raise ValueError(f"{what} must be contiguous [{D}], got shape {tuple(p.shape)}")
        if p_type is not None and p.dtype != p_type:
            raise ValueError(f"weight and bias must have one type, got {p_type} and {p.dtype}")
        p_type = p.dtype
    return x.numel() // D, D, p_type or x.dtype


def _out_dtype(x, out_dtype):
    if out_dtype is None or out_dtype == x.dtype:
        return x.dtype
    if out_dtype not in TYPES or x.dtype != torch.float32:
        raise ValueError(f"out_dtype {out_dtype} is not available from {x.dtype}: the type of x, or a 16-bit type "
                         "from float32")
    return out_dtype


def _ptr(t):
    return 0 if t is None else t.data_ptr()


def _on_device(x):
    return x.get_device() == _current_device()


def _result(x, dtype):
    """A contiguous tensor of x's shape."""
    if dtype == x.dtype and x.is_contiguous():
        return torch.empty_like(x)
    return torch.empty(x.shape, dtype=dtype, device=x.device)


def cce_layer_norm_forward(x, weight=None, bias=None, eps=1e-5, *, out_dtype=None, stats=True, stream=None):
    """(y, mean, rstd) of a layer norm over the last dimension; mean and rstd
    are fp32 with one value a row, None with stats=False."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return cce_layer_norm_forward(x, weight, bias, eps, out_dtype=out_dtype, stats=stats)
    N, D, p_type = _check(x, weight, bias)
    y_type = _out_dtype(x, out_dtype)
    if not _on_device(x):
        with torch.cuda.device(x.device):
            return cce_layer_norm_forward(x, weight, bias, eps, out_dtype=out_dtype, stats=stats)
    dev = x.device
    x, inner, row, outer = _rows(x)
    y = _result(x, y_type)
    mean = torch.empty(N, dtype=torch.float32, device=dev) if stats else None
    rstd = torch.empty(N, dtype=torch.float32, device=dev) if stats else None
    st = _layer_forward(x.data_ptr(), inner, row, outer, TYPES[x.dtype], _ptr(weight), _ptr(bias), TYPES[p_type], N,
                        D, eps, y.data_ptr(), TYPES[y_type], _ptr(mean), _ptr(rstd), _raw_stream(x.get_device()))
    if st:
        _lib.check(st, "cce_layer_norm_forward")
    return y, mean, rstd


def cce_rms_norm_forward(x, weight=None, eps=1e-6, *, weight_offset=0.0, out_dtype=None, stats=True, stream=None):
    """(y, rstd) of an RMS norm over the last dimension: y = x * rstd *
    (weight_offset + weight); rstd is None with stats=False."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return cce_rms_norm_forward(x, weight, eps, weight_offset=weight_offset, out_dtype=out_dtype, stats=stats)
    N, D, p_type = _check(x, weight, None)
    y_type = _out_dtype(x, out_dtype)
    if not _on_device(x):
        with torch.cuda.device(x.device):
            return cce_rms_norm_forward(x, weight, eps, weight_offset=weight_offset, out_dtype=out_dtype, stats=stats)
    dev = x.device
    x, inner, row, outer = _rows(x)
    y = _result(x, y_type)
    rstd = torch.empty(N, dtype=torch.float32, device=dev) if stats else None
    st = _rms_forward(x.data_ptr(), inner, row, outer, TYPES[x.dtype], _ptr(weight), TYPES[p_type], weight_offset, N,
                      D, eps, y.data_ptr(), TYPES[y_type], _ptr(rstd), _raw_stream(x.get_device()))
    if st:
        _lib.check(st, "cce_rms_norm_forward")
    return y, rstd


def _check_backward(grad_y, x, N, stats):
    if grad_y.get_device() != x.get_device():
        raise ValueError(f"grad_y must be on {x.device}, got {grad_y.device}")
    if grad_y.shape != x.shape:
        raise ValueError(f"grad_y must have the shape of x, {tuple(x.shape)}, got {tuple(grad_y.shape)}")
    if grad_y.dtype != x.dtype and (x.dtype != torch.float32 or grad_y.dtype not in TYPES):
        raise ValueError(f"grad_y must be {x.dtype}, or a 16-bit type for float32 x, got {grad_y.dtype}")
    for what, s in stats:
        if s.get_device() != x.get_device() or s.dtype != torch.float32 or s.numel() != N or not s.is_contiguous():
            raise ValueError(f"{what} must be contiguous float32 with {N} values on {x.device}")


def cce_layer_norm_backward(grad_y, x, weight, mean, rstd, *, need_dx=True, need_dweight=True, need_dbias=True,
                            param_dtype=None, stream=None):
    """(dx, dweight, dbias) of a layer norm whose forward gave mean and rstd;
    None for those not needed.  The parameters' gradients have the weight's
    type, or param_dtype where there is no weight (x's type if not given)."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return cce_layer_norm_backward(grad_y, x, weight, mean, rstd, need_dx=need_dx, need_dweight=need_dweight,
                                           need_dbias=need_dbias, param_dtype=param_dtype)
    N, D, p_type = _check(x, weight, None)
    if weight is None and param_dtype is not None:
        if param_dtype not in TYPES:
            raise ValueError(f"param_dtype must be bfloat16, float16 or float32, got {param_dtype}")
        p_type = param_dtype
    _check_backward(grad_y, x, N, (("mean", mean), ("rstd", rstd)))
    if not _on_device(x):
        with torch.cuda.device(x.device):
            return cce_layer_norm_backward(grad_y, x, weight, mean, rstd, need_dx=need_dx, need_dweight=need_dweight,
                                           need_dbias=need_dbias, param_dtype=param_dtype)
    dev = x.device
    x, xi, xr, xo = _rows(x)
    grad_y, gi, gr, go = _rows(grad_y)
    dx = _result(x, x.dtype) if need_dx else None
    dw = torch.empty(D, dtype=p_type, device=dev) if need_dweight else None
    db = torch.empty(D, dtype=p_type, device=dev) if need_dbias else None
    need = _workspace_bytes(N, D) if need_dweight or need_dbias else 0
    ws = torch.empty(need, dtype=torch.uint8, device=dev) if need else None
    st = _layer_backward(grad_y.data_ptr(), gi, gr, go, TYPES[grad_y.dtype], x.data_ptr(), xi, xr, xo, TYPES[x.dtype],
                         _ptr(weight), TYPES[p_type], mean.data_ptr(), rstd.data_ptr(), N, D, _ptr(dx), _ptr(dw),
                         _ptr(db), _ptr(ws), need, _raw_stream(x.get_device()))
    if st:
        _lib.check(st, "cce_layer_norm_backward")
    return dx, dw, db


def cce_rms_norm_backward(grad_y, x, weight, rstd, *, weight_offset=0.0, need_dx=True, need_dweight=True,
                          stream=None):
    """(dx, dweight) of an RMS norm whose forward gave rstd; None for those
    not needed (dweight also where there is no weight)."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return cce_rms_norm_backward(grad_y, x, weight, rstd, weight_offset=weight_offset, need_dx=need_dx,
                                         need_dweight=need_dweight)
    N, D, p_type = _check(x, weight, None)
    _check_backward(grad_y, x, N, (("rstd", rstd),))
    if not _on_device(x):
        with torch.cuda.device(x.device):
            return cce_rms_norm_backward(grad_y, x, weight, rstd, weight_offset=weight_offset, need_dx=need_dx,
                                         need_dweight=need_dweight)
    dev = x.device
    x, xi, xr, xo = _rows(x)
    grad_y, gi, gr, go = _rows(grad_y)
    dx = _result(x, x.dtype) if need_dx else None
    dw = torch.empty(D, dtype=p_type, device=dev) if need_dweight and weight is not None else None
    need = _workspace_bytes(N, D) if dw is not None else 0
    ws = torch.empty(need, dtype=torch.uint8, device=dev) if need else None
    st = _rms_backward(grad_y.data_ptr(), gi, gr, go, TYPES[grad_y.dtype], x.data_ptr(), xi, xr, xo, TYPES[x.dtype],
                       _ptr(weight), TYPES[p_type], weight_offset, rstd.data_ptr(), N, D, _ptr(dx), _ptr(dw),
                       _ptr(ws), need, _raw_stream(x.get_device()))
    if st:
        _lib.check(st, "cce_rms_norm_backward")
    return dx, dw


class LayerNormFunction(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias, eps, out_dtype):
        y, mean, rstd = cce_layer_norm_forward(x, weight, bias, eps, out_dtype=out_dtype)
        ctx.save_for_backward(x, weight, mean, rstd)
        ctx.param_dtype = None if bias is None else bias.dtype
        return y

    @staticmethod
    @once_differentiable
    def backward(ctx, grad_y):
        x, weight, mean, rstd = ctx.saved_tensors
        need = ctx.needs_input_grad
        dx, dw, db = cce_layer_norm_backward(grad_y, x, weight, mean, rstd, need_dx=need[0], need_dweight=need[1],
                                             need_dbias=need[2], param_dtype=ctx.param_dtype)
        return dx, dw, db, None, None


class RMSNormFunction(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, eps, weight_offset, out_dtype):
        y, rstd = cce_rms_norm_forward(x, weight, eps, weight_offset=weight_offset, out_dtype=out_dtype)
        ctx.save_for_backward(x, weight, rstd)
        ctx.weight_offset = weight_offset
        return y

    @staticmethod
    @once_differentiable
    def backward(ctx, grad_y):
        x, weight, rstd = ctx.saved_tensors
        need = ctx.needs_input_grad
        dx, dw = cce_rms_norm_backward(grad_y, x, weight, rstd, weight_offset=ctx.weight_offset, need_dx=need[0],
                                       need_dweight=need[1])
        return dx, dw, None, None, None


def layer_norm(x, weight=None, bias=None, eps=1e-5, out_dtype=None):
    """Layer norm over x's last dimension: (x - mean) / sqrt(var + eps) *
    weight + bias, differentiable in x, weight and bias (once).

    weight and bias [D] are optional and share one type, which may differ from
    x's.  out_dtype: a 16-bit result from float32 rows (default: x's type)."""
    if torch.is_grad_enabled() and (x.requires_grad or (weight is not None and weight.requires_grad)
                                    or (bias is not None and bias.requires_grad)):
        return LayerNormFunction.apply(x, weight, bias, eps, out_dtype)
    return cce_layer_norm_forward(x, weight, bias, eps, out_dtype=out_dtype, stats=False)[0]


def rms_norm(x, weight=None, eps=1e-6, weight_offset=0.0, out_dtype=None):
    """RMS norm over x's last dimension: x / sqrt(mean(x^2) + eps) *
    (weight_offset + weight), differentiable in x and weight (once).

    weight_offset is 1 for models that store the weight minus one (without a
    weight there is no factor).  out_dtype as for layer_norm."""
    if torch.is_grad_enabled() and (x.requires_grad or (weight is not None and weight.requires_grad)):
        return RMSNormFunction.apply(x, weight, eps, weight_offset, out_dtype)
    return cce_rms_norm_forward(x, weight, eps, weight_offset=weight_offset, out_dtype=out_dtype, stats=False)[0]
