"""ctypes binding of libcce.so (declarations in include/cce*.h).

Loading fails loudly when the library has not been built: there is no
fallback implementation.
"""
from __future__ import annotations

import ctypes
import os

import torch  # noqa: F401  (loads the CUDA runtime libcce.so links against)

from . import build

NATIVE_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "_native.so")
LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libcce.so")

CCE_OK = 0
STATUS_NAMES = {
    0: "CCE_OK", 1: "CCE_ERR_NULL", 2: "CCE_ERR_SHAPE", 3: "CCE_ERR_ALIGN", 4: "CCE_ERR_ARG",
    5: "CCE_ERR_WORKSPACE", 6: "CCE_ERR_DEVICE", 7: "CCE_ERR_CUDA", 8: "CCE_ERR_TARGET_RANGE",
    9: "CCE_ERR_TIMEOUT",
}
RED = {"none": 0, "sum": 1, "mean": 2}
DEVERR_TARGET_RANGE = 1
DEVERR_TIMEOUT = 2
NUM_PHASES = 8
SORT_VOCAB = 4
FWD_SKIP_IGNORED = 1


class CCEError(RuntimeError):
    def __init__(self, status: int, what: str = ""):
        self.status = status
        name = STATUS_NAMES.get(status, str(status))
        super().__init__(f"{what}: {name}" if what else name)


class MemoryReport(ctypes.Structure):
    _fields_ = [
        ("logits_fp32_bytes", ctypes.c_uint64),
        ("dE_bytes", ctypes.c_uint64),
        ("dC_bytes", ctypes.c_uint64),
        ("lse_bytes", ctypes.c_uint64),
        ("fwd_workspace_bytes", ctypes.c_uint64),
        ("bwd_workspace_bytes", ctypes.c_uint64),
        ("bwd_chunk_cols", ctypes.c_uint64),
        ("fwd_vocab_splits", ctypes.c_uint64),
    ]


class Strided(ctypes.Structure):
    """cce_strided of include/cce_ops.h."""
    _fields_ = [("in_", ctypes.c_void_p), ("out", ctypes.c_void_p), ("in_type", ctypes.c_int32),
                ("out_type", ctypes.c_int32), ("size", ctypes.c_int64 * 4), ("in_stride", ctypes.c_int64 * 4),
                ("out_stride", ctypes.c_int64 * 4)]


class RowCopy(ctypes.Structure):
    """cce_row_copy of include/cce_layers.h."""
    _fields_ = [("src", ctypes.c_void_p), ("dst", ctypes.c_void_p), ("inner", ctypes.c_int64),
                ("row_stride", ctypes.c_int64), ("outer_stride", ctypes.c_int64), ("pitch", ctypes.c_int64),
                ("rows", ctypes.c_int64), ("cols", ctypes.c_int64), ("bytes", ctypes.c_int32)]


class AdamWTensor(ctypes.Structure):
    """cce_adamw_tensor of include/cce_optim.h."""
    _fields_ = [("grad", ctypes.c_void_p), ("param", ctypes.c_void_p), ("master", ctypes.c_void_p),
                ("exp_avg", ctypes.c_void_p), ("exp_avg_sq", ctypes.c_void_p), ("exp_avg_scale", ctypes.c_void_p),
                ("rms_scale", ctypes.c_void_p), ("n", ctypes.c_int64), ("grad_type", ctypes.c_int32),
                ("param_type", ctypes.c_int32), ("weight_decay", ctypes.c_float)]


class AdamWOptions(ctypes.Structure):
    """cce_adamw_options of include/cce_optim.h."""
    _fields_ = [("lr", ctypes.c_double), ("beta1", ctypes.c_double), ("beta2", ctypes.c_double),
                ("eps", ctypes.c_double), ("step", ctypes.c_int64), ("step_ptr", ctypes.c_void_p),
                ("lr_ptr", ctypes.c_void_p), ("norm", ctypes.c_void_p), ("max_norm", ctypes.c_float),
                ("eps_norm", ctypes.c_float), ("seed", ctypes.c_uint32)]


_lib = None


def load() -> ctypes.CDLL:
    global _lib
    if _lib is not None:
        return _lib
    for path in (LIB_PATH, NATIVE_PATH):
        if os.path.exists(path):
            continue
        raise ImportError(f"{path} is not built; run `{build.COMMAND}` (there is no non-CUDA fallback)")
    if build.built_for() not in ("", build.versions()):
        raise ImportError(f"{NATIVE_PATH} was built for {build.built_for()}, and this is {build.versions()}; run "
                          f"`{build.COMMAND}`")
    lib = ctypes.CDLL(LIB_PATH)
    vp, i64, sz = ctypes.c_void_p, ctypes.c_int64, ctypes.c_size_t
    lib.cce_forward_workspace_bytes.argtypes = [i64, i64, i64]
    lib.cce_forward_workspace_bytes.restype = sz
    lib.cce_backward_workspace_bytes.argtypes = [i64, i64, i64]
    lib.cce_backward_workspace_bytes.restype = sz
    lib.cce_forward.argtypes = [vp, vp, vp, i64, i64, i64, i64, ctypes.c_int, vp, vp, vp, sz, vp, vp]
    lib.cce_forward.restype = ctypes.c_int
    lib.cce_backward.argtypes = [vp, vp, vp, vp, vp, i64, i64, i64, i64, ctypes.c_int, ctypes.c_float,
                                 vp, vp, vp, sz, vp, vp, vp]
    lib.cce_backward.restype = ctypes.c_int
    lib.cce_forward_ex.argtypes = [vp, vp, vp, i64, i64, i64, i64, ctypes.c_int, ctypes.c_float, vp, vp, vp, sz,
                                   vp, vp]
    lib.cce_forward_ex.restype = ctypes.c_int
    lib.cce_backward_ex.argtypes = [vp, vp, vp, vp, vp, i64, i64, i64, i64, ctypes.c_int, ctypes.c_float,
                                    ctypes.c_float, ctypes.c_int, vp, vp, vp, sz, vp, vp, vp]
    lib.cce_backward_ex.restype = ctypes.c_int
    lib.cce_backward_workspace_bytes_ex.argtypes = [i64, i64, i64, ctypes.c_int]
    lib.cce_backward_workspace_bytes_ex.restype = sz
    lib.cce_backward_ex2.argtypes = [vp, vp, vp, vp, vp, i64, i64, i64, i64, ctypes.c_int, ctypes.c_float,
                                     ctypes.c_float, ctypes.c_int, sz, vp, vp, vp, sz, vp, vp, vp]
    lib.cce_backward_ex2.restype = ctypes.c_int
    lib.cce_backward_workspace_bytes_ex2.argtypes = [i64, i64, i64, ctypes.c_int, sz]
    lib.cce_backward_workspace_bytes_ex2.restype = sz
    lib.cce_backward_chunk_cols.argtypes = [i64, i64, sz]
    lib.cce_backward_chunk_cols.restype = ctypes.c_uint64
    lib.cce_vocab_sort_workspace_bytes.argtypes = [i64, i64, i64]
    lib.cce_vocab_sort_workspace_bytes.restype = sz
    lib.cce_vocab_logit_sums.argtypes = [vp, vp, vp, i64, i64, i64, i64, vp, vp, sz, vp]
    lib.cce_vocab_logit_sums.restype = ctypes.c_int
    lib.cce_vocab_order.argtypes = [vp, i64, vp, vp, sz, vp]
    lib.cce_vocab_order.restype = ctypes.c_int
    lib.cce_forward_workspace_bytes_ex.argtypes = [i64, i64, i64, ctypes.c_int]
    lib.cce_forward_workspace_bytes_ex.restype = sz
    lib.cce_forward_ex2.argtypes = [vp, vp, vp, i64, i64, i64, i64, ctypes.c_int, ctypes.c_float, ctypes.c_int, vp,
                                    vp, vp, sz, vp, vp]
    lib.cce_forward_ex2.restype = ctypes.c_int
    lib.cce_loss_and_grad_workspace_bytes.argtypes = [i64, i64, i64, sz]
    lib.cce_loss_and_grad_workspace_bytes.restype = sz
    lib.cce_loss_and_grad.argtypes = [vp, vp, vp, i64, i64, i64, i64, ctypes.c_int, ctypes.c_float, ctypes.c_float,
                                      ctypes.c_int, sz, vp, vp, vp, vp, vp, sz, vp, vp, vp]
    lib.cce_loss_and_grad.restype = ctypes.c_int
    lib.cce_scale_grads.argtypes = [vp, i64, vp, i64, vp, vp]
    lib.cce_scale_grads.restype = ctypes.c_int
    lib.cce_forward_noalloc.argtypes = [vp, vp, vp, i64, i64, i64, i64, ctypes.c_int, vp, vp, vp, vp]
    lib.cce_forward_noalloc.restype = ctypes.c_int
    lib.cce_selftest_wait_timeout.argtypes = [vp, ctypes.c_uint32, vp]
    lib.cce_selftest_wait_timeout.restype = ctypes.c_int
    lib.cce_selftest_pair_timeout.argtypes = [vp, ctypes.c_uint32, ctypes.c_int, vp]
    lib.cce_selftest_pair_timeout.restype = ctypes.c_int
    lib.cce_selftest_pair_map_words.argtypes = [ctypes.c_int]
    lib.cce_selftest_pair_map_words.restype = ctypes.c_int
    lib.cce_selftest_grad_layout.argtypes = [ctypes.c_int]
    lib.cce_selftest_grad_layout.restype = ctypes.c_int
    lib.cce_memory_accounting.argtypes = [i64, i64, i64, ctypes.POINTER(MemoryReport)]
    lib.cce_memory_accounting.restype = ctypes.c_int
    lib.cce_status_string.argtypes = [ctypes.c_int]
    lib.cce_status_string.restype = ctypes.c_char_p
    lib.cce_abi_version.argtypes = []
    lib.cce_abi_version.restype = ctypes.c_int
    lib.cce_kernel_launch_count.argtypes = []
    lib.cce_kernel_launch_count.restype = ctypes.c_uint64
    lib.cce_profile_enable.argtypes = [ctypes.c_int]
    lib.cce_profile_enable.restype = ctypes.c_int
    lib.cce_profile_reset.argtypes = []
    lib.cce_profile_reset.restype = ctypes.c_int
    lib.cce_profile_read.argtypes = [ctypes.POINTER(ctypes.c_double), ctypes.POINTER(ctypes.c_int64)]
    lib.cce_profile_read.restype = ctypes.c_int
    lib.cce_profile_phase_name.argtypes = [ctypes.c_int]
    lib.cce_profile_phase_name.restype = ctypes.c_char_p
    # include/cce_ops.h
    rows = [i64, i64, i64]  # inner, row stride, outer stride
    ci, cf = ctypes.c_int, ctypes.c_float
    lib.cce_ops_abi_version.argtypes = []
    lib.cce_ops_abi_version.restype = ci
    lib.cce_layer_norm_forward.argtypes = [vp] + rows + [ci, vp, vp, ci, i64, i64, cf, vp, ci, vp, vp, vp]
    lib.cce_layer_norm_forward.restype = ci
    lib.cce_rms_norm_forward.argtypes = [vp] + rows + [ci, vp, ci, cf, i64, i64, cf, vp, ci, vp, vp]
    lib.cce_rms_norm_forward.restype = ci
    lib.cce_layer_norm_backward.argtypes = ([vp] + rows + [ci, vp] + rows
                                            + [ci, vp, ci, vp, vp, i64, i64, vp, vp, vp, vp, sz, vp])
    lib.cce_layer_norm_backward.restype = ci
    lib.cce_rms_norm_backward.argtypes = ([vp] + rows + [ci, vp] + rows
                                          + [ci, vp, ci, cf, vp, i64, i64, vp, vp, vp, sz, vp])
    lib.cce_rms_norm_backward.restype = ci
    lib.cce_norm_backward_workspace_bytes.argtypes = [i64, i64]
    lib.cce_norm_backward_workspace_bytes.restype = sz
    lib.cce_grad_norm.argtypes = [vp, i64, vp, i64, ci, vp, vp, sz, vp]
    lib.cce_grad_norm.restype = ci
    lib.cce_clip_grads.argtypes = [vp, i64, vp, i64, ci, cf, cf, vp, vp, sz, vp]
    lib.cce_clip_grads.restype = ci
    lib.cce_grad_norm_workspace_bytes.argtypes = [i64, i64]
    lib.cce_grad_norm_workspace_bytes.restype = sz
    # include/cce_layers.h
    lib.cce_layers_abi_version.argtypes = []
    lib.cce_layers_abi_version.restype = ci
    mat = [vp, i64]  # pointer, pitch
    lib.cce_linear_forward.argtypes = (mat + mat + [ci, vp, ci, vp, i64, i64, i64] + [ci, i64, i64, i64] + mat + [ci] + mat
                                       + [ci, vp, sz, vp])
    lib.cce_linear_backward.argtypes = (mat + [ci] + mat + mat + [ci] + mat + [ci, ci, i64, i64, i64, vp, vp, vp, ci, vp,
                                                                               sz, vp])
    lib.cce_gated_linear_forward.argtypes = (mat + mat + mat + [ci, ci, i64, i64, i64] + mat
                                             + [vp, vp, i64, ci, vp, sz, vp])
    lib.cce_gated_linear_backward.argtypes = (mat * 4 + [ci] + mat + mat + [ci, ci, i64, i64, i64, vp, vp, vp, vp, sz, vp])
    lib.cce_layers_take_error.argtypes = [vp, vp]
    lib.cce_copy_rows.argtypes = [ctypes.POINTER(RowCopy), ci, vp]
    for name in ("cce_linear_forward", "cce_linear_backward", "cce_gated_linear_forward", "cce_gated_linear_backward",
                 "cce_layers_take_error", "cce_copy_rows"):
        getattr(lib, name).restype = ci
    for name in ("linear_forward", "linear_backward", "gated_linear_forward", "gated_linear_backward"):
        query = getattr(lib, f"cce_{name}_workspace_bytes")
        query.argtypes = [i64, i64, i64]
        query.restype = sz
    # include/cce_layers_ex.h
    lib.cce_layers_plan_searches.argtypes = []
    lib.cce_layers_plan_searches.restype = ctypes.c_uint64
    for name in ("linear_backward", "gated_linear_backward"):
        query = getattr(lib, f"cce_{name}_workspace_bytes_ex")
        query.argtypes = [i64, i64, i64, ci]
        query.restype = sz
    lib.cce_selftest_layers_wait_timeout.argtypes = [ctypes.c_uint32, vp]
    lib.cce_selftest_layers_wait_timeout.restype = ci
    # include/cce_optim.h
    lib.cce_optim_abi_version.argtypes = []
    lib.cce_optim_abi_version.restype = ci
    lib.cce_adamw_step.argtypes = [ctypes.POINTER(AdamWTensor), i64, ci, ctypes.POINTER(AdamWOptions), vp]
    lib.cce_adamw_step.restype = ci
    _lib = lib
    return lib


def check(status: int, what: str = "") -> None:
    if status != CCE_OK:
        raise CCEError(status, what)
