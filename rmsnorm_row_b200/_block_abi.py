"""ctypes view of include/block_ops.h, and the extension behind the package's tensor-level
functions. The library is the one of ``_abi``; loading either fails loudly when it has not been
built."""
from __future__ import annotations

import ctypes
from . import _abi
from ._abi import fn_operand

BO_BF16, BO_FP16, BO_E4M3, BO_FP32 = 0, 1, 2, 3

_int, _i64, _ptr, _dbl = ctypes.c_int, ctypes.c_int64, ctypes.c_void_p, ctypes.c_double


class nq_config(ctypes.Structure):
    _fields_ = [("D", _int), ("is_rms", _int), ("has_residual", _int), ("has_gate", _int),
                ("has_weight", _int), ("has_bias", _int), ("affine_fp32", _int),
                ("has_modulation", _int), ("eps", _dbl)]


class nq_args(ctypes.Structure):
    _fields_ = [("B", _i64), ("L", _i64), ("tokens_per_frame", _i64),
                ("x", fn_operand), ("residual", fn_operand), ("gate", fn_operand),
                ("scale", fn_operand), ("shift", fn_operand),
                ("weight", _ptr), ("bias", _ptr),
                ("q", _ptr), ("q_stride_b", _i64), ("q_stride_l", _i64),
                ("row_scale", _ptr),
                ("r", _ptr), ("r_stride_b", _i64), ("r_stride_l", _i64)]


c_int4 = _int * 4


class rn_config(ctypes.Structure):
    _fields_ = [("dtype", _int), ("heads", _int), ("head_dim", _int), ("axes", _int), ("section", c_int4),
                ("norm", _int), ("has_weight", _int), ("weight_fp32", _int), ("half_pairs", _int),
                ("shared_frequencies", _int), ("index64", _int), ("theta", _dbl), ("eps", _dbl)]


class rn_rows(ctypes.Structure):
    _fields_ = [("ptr", _ptr), ("stride_b", _i64), ("stride_l", _i64), ("stride_h", _i64)]


class rn_args(ctypes.Structure):
    _fields_ = [("B", _i64), ("L", _i64), ("x", rn_rows), ("positions", _ptr), ("pos_stride_b", _i64),
                ("pos_stride_l", _i64), ("weight", _ptr), ("y", rn_rows)]


class rn_backward_args(ctypes.Structure):
    _fields_ = [("B", _i64), ("L", _i64), ("grad", rn_rows), ("x", rn_rows), ("positions", _ptr),
                ("pos_stride_b", _i64), ("pos_stride_l", _i64), ("weight", _ptr), ("dx", rn_rows),
                ("dweight", _ptr), ("workspace", _ptr), ("workspace_bytes", ctypes.c_uint64)]


class lg_config(ctypes.Structure):
    _fields_ = [("dtype", _int), ("K", _i64), ("N", _i64), ("act", _int), ("has_bias", _int), ("has_gate", _int),
                ("has_residual", _int)]


class lg_args(ctypes.Structure):
    _fields_ = [("B", _i64), ("L", _i64), ("tokens_per_frame", _i64), ("x", fn_operand), ("weight", _ptr),
                ("weight_stride", _i64), ("bias", _ptr), ("gate", fn_operand), ("residual", fn_operand),
                ("x_scale", _ptr), ("weight_scale", _ptr), ("out", _ptr), ("out_stride_b", _i64),
                ("out_stride_l", _i64)]


# operator -> (config, {launch and its validate: args})
OPERATORS = {
    "norm_quant": (nq_config, {"launch": nq_args}),
    "rope_norm": (rn_config, {"launch": rn_args, "backward_launch": rn_backward_args}),
    "linear_gate": (lg_config, {"launch": lg_args}),
}
EXPORTED = tuple(f"{op}_{call}" for op, (_, calls) in OPERATORS.items()
                 for name in calls for call in (name, name.replace("launch", "validate"))) + tuple(
    f"{op}_{call}" for op in OPERATORS for call in ("create", "destroy")) + (
    "rope_norm_backward_workspace", "linear_gate_timeouts", "block_ops_status_string", "block_ops_last_cuda_error")

_declared = None


def load() -> ctypes.CDLL:
    """The loaded library with the prototypes of include/block_ops.h."""
    global _declared
    if _declared is None:
        lib = _abi.load()
        P = ctypes.POINTER
        for op, (config, calls) in OPERATORS.items():
            getattr(lib, f"{op}_create").argtypes = [P(_ptr), P(config)]
            getattr(lib, f"{op}_destroy").argtypes = [_ptr]
            for name, args in calls.items():
                getattr(lib, f"{op}_{name}").argtypes = [_ptr, P(args), _ptr]
                getattr(lib, f"{op}_{name.replace('launch', 'validate')}").argtypes = [_ptr, P(args)]
        lib.rope_norm_backward_workspace.argtypes = [_ptr, _i64, _i64, P(ctypes.c_uint64)]
        lib.linear_gate_timeouts.argtypes = [P(_int)]
        for name in EXPORTED:
            getattr(lib, name).restype = _int
        lib.block_ops_status_string.argtypes = [_int]
        lib.block_ops_status_string.restype = ctypes.c_char_p
        lib.block_ops_last_cuda_error.argtypes = []
        lib.block_ops_last_cuda_error.restype = _int
        _declared = lib
    return _declared


def check(status: int, what: str) -> None:
    """Raises FusedNormError for any status but FN_OK."""
    if status == _abi.FN_OK:
        return
    detail = load().block_ops_status_string(status).decode()
    if status == _abi.FN_ERR_CUDA:
        detail += f" (cudaError {load().block_ops_last_cuda_error()})"
    raise _abi.FusedNormError(status, what, detail)


_binding = None


def binding():
    """The extension behind norm_quant, rope and linear (csrc/binding)."""
    global _binding
    if _binding is None:
        _abi.load()
        try:
            from . import _binding as module
        except ImportError as e:
            raise ImportError("rmsnorm_row_b200/_binding.so does not load: build it with `python -m rmsnorm_row_b200.build` "
                              f"(there is no fallback implementation): {e}") from e
        _binding = module
    return _binding
