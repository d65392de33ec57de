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
of 16 up to 16384, and scale and shift may both be None (no modulation). The functions are not
recorded by autograd: their results require no gradient, whatever their inputs do.
"""
from __future__ import annotations

from typing import Optional

import torch

from ._block_abi import binding


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
    return binding().norm_quant(residual, x, gate, weight, bias, scale, shift, norm_type, eps, out, row_scale_out,
                                residual_out, stream)


def norm_scale_shift_quant(x: torch.Tensor, weight: Optional[torch.Tensor], bias: Optional[torch.Tensor],
                           scale: Optional[torch.Tensor], shift: Optional[torch.Tensor],
                           norm_type: str = "layer", eps: float = 1e-6, *,
                           out: Optional[torch.Tensor] = None,
                           row_scale_out: Optional[torch.Tensor] = None,
                           stream: Optional[torch.cuda.Stream] = None):
    """(q, row_scale) of the normed, modulated, quantised rows of x (no residual)."""
    return binding().norm_quant(None, x, None, weight, bias, scale, shift, norm_type, eps, out, row_scale_out, None,
                                stream)
