"""Norm rows with an e4m3 output and one scale per row (include/block_ops.h, norm_quant).

The two ops take the arguments of ``fused_residual_norm_scale_shift`` and
``norm_scale_shift``, in their order, and return e4m3 rows with their scales in the place of
y, which is what ``linear_gate_residual`` takes as x and x_scale:

    fused_residual_norm_scale_shift_quant(residual, x, gate, weight, bias, scale, shift,
                                          norm_type, eps) -> (q, row_scale, r)
    norm_scale_shift_quant(x, weight, bias, scale, shift, norm_type, eps) -> (q, row_scale)

    y = norm(r) (* weight + bias) (* (1 + scale) + shift)        not rounded
    row_scale = max |y| / 448 over the row (1 for a row of zeros)
    q = e4m3(y / row_scale)

Operand shapes, dtypes, streams and devices are those of the 16-bit ops; D may be any multiple
of 16 up to 16384, and scale and shift may both be None (no modulation).
"""
from __future__ import annotations

from typing import Optional

import torch

from . import _abi, _block_abi
from .api import _affine_fp32, _check_tensor, _norm_flag, _operand, _vector


def _rows(t: torch.Tensor, B: int, L: int) -> _abi.fn_operand:
    s = t.stride()
    return _abi.fn_operand(t.data_ptr(), s[0] if B > 1 else 0, 0, s[1] if L > 1 else 0)


def _out(t: torch.Tensor, name: str, shape, dtype, device) -> torch.Tensor:
    if not isinstance(t, torch.Tensor) or t.dtype != dtype or tuple(t.shape) != tuple(shape) or t.device != device:
        raise ValueError(f"{name} must be a {dtype} tensor of shape {tuple(shape)} on {device}")
    return t


def _quant(residual, x, gate, weight, bias, scale, shift, norm_type, eps, out, row_scale_out, residual_out, stream):
    if not isinstance(x, torch.Tensor) or x.dim() != 3:
        raise ValueError("x must be a (B, L, D) tensor")
    device = x.device
    if device.type != "cuda":
        raise ValueError("x must be a CUDA tensor")
    _check_tensor(x, "x", device)
    B, L, D = x.shape
    if D % 16 or not 16 <= D <= 16384:
        raise ValueError(f"D must be a multiple of 16 from 16 to 16384, got {D}")
    if (scale is None) != (shift is None):
        raise ValueError("scale and shift come together")
    if eps < 0:
        raise ValueError("eps must not be negative")
    is_rms, f32 = _norm_flag(norm_type), _affine_fp32(weight, bias)
    a = _block_abi.nq_args(B=B, L=L)
    a.x = _rows(x, B, L)
    frames = set()
    for name, t in (("gate", gate), ("scale", scale), ("shift", shift)):
        if t is not None:
            op, F = _operand(t, name, B, L, D, device)
            setattr(a, name, op)
            if F:
                frames.add(F)
    if len(frames) > 1:
        raise ValueError(f"operands disagree on the frame count: {sorted(frames)}")
    if frames:
        a.tokens_per_frame = L // frames.pop()
    a.weight = _vector(weight, "weight", D, device)
    a.bias = _vector(bias, "bias", D, device)
    r = None
    if residual is not None:
        _check_tensor(residual, "residual", device)
        if residual.shape != x.shape:
            raise ValueError("residual must match x")
        a.residual = _rows(residual, B, L)
        r = torch.empty((B, L, D), dtype=x.dtype, device=device) if residual_out is None else residual_out
        _check_tensor(_out(r, "residual_out", x.shape, x.dtype, device), "residual_out", device)
        a.r, (a.r_stride_b, a.r_stride_l) = r.data_ptr(), r.stride()[:2]
    if out is None:
        out = torch.empty((B, L, D), dtype=torch.float8_e4m3fn, device=device)
    elif _out(out, "out", x.shape, torch.float8_e4m3fn, device).stride(-1) != 1:
        raise ValueError("out needs a contiguous channel dimension")
    if row_scale_out is None:
        row_scale_out = torch.empty((B, L), dtype=torch.float32, device=device)
    elif not _out(row_scale_out, "row_scale_out", (B, L), torch.float32, device).is_contiguous():
        raise ValueError("row_scale_out must be contiguous")
    a.q, (a.q_stride_b, a.q_stride_l) = out.data_ptr(), out.stride()[:2]
    a.row_scale = row_scale_out.data_ptr()
    key = (D, is_rms, residual is not None, gate is not None, weight is not None, bias is not None, f32,
           scale is not None, float(eps))
    h = _block_abi.handle("norm_quant", key, lambda: _block_abi.nq_config(*(int(v) for v in key[:-1]), key[-1]))
    _block_abi.launch("norm_quant", h, a, device, stream)
    return out, row_scale_out, r


def fused_residual_norm_scale_shift_quant(residual: torch.Tensor, x: torch.Tensor,
                                          gate: Optional[torch.Tensor], weight: Optional[torch.Tensor],
                                          bias: Optional[torch.Tensor], scale: Optional[torch.Tensor],
                                          shift: Optional[torch.Tensor], norm_type: str = "layer",
                                          eps: float = 1e-6, *, out: Optional[torch.Tensor] = None,
                                          row_scale_out: Optional[torch.Tensor] = None,
                                          residual_out: Optional[torch.Tensor] = None,
                                          stream: Optional[torch.cuda.Stream] = None):
    """(q, row_scale, r) of r = residual + gate * x and its normed, modulated, quantised rows.

    `residual_out` may be `residual` itself (in-place residual update).
    """
    if residual is None:
        raise ValueError("residual is required (norm_scale_shift_quant has none)")
    return _quant(residual, x, gate, weight, bias, scale, shift, norm_type, eps, out, row_scale_out,
                  residual_out, stream)


def norm_scale_shift_quant(x: torch.Tensor, weight: Optional[torch.Tensor], bias: Optional[torch.Tensor],
                           scale: Optional[torch.Tensor], shift: Optional[torch.Tensor],
                           norm_type: str = "layer", eps: float = 1e-6, *,
                           out: Optional[torch.Tensor] = None,
                           row_scale_out: Optional[torch.Tensor] = None,
                           stream: Optional[torch.cuda.Stream] = None):
    """(q, row_scale) of the normed, modulated, quantised rows of x (no residual)."""
    return _quant(None, x, None, weight, bias, scale, shift, norm_type, eps, out, row_scale_out, None, stream)[:2]
