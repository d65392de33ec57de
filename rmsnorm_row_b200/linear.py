"""Matrix product with bias, activation, gate and residual in its epilogue
(include/block_ops.h, linear_gate).

    linear_gate_residual(x, weight, bias=None, gate=None, residual=None, *, activation="none",
                         x_scale=None, weight_scale=None) -> out
    out = residual + gate * activation(x @ weight.T + bias)

x is (B, L, K) and weight (N, K), both bf16, fp16 or e4m3, with contiguous last dimensions;
out is (B, L, N) in x's type, or bf16 for e4m3. e4m3 needs x_scale (B, L), as
``norm_scale_shift_quant`` returns it, and weight_scale (N,), both fp32: the product is that of
x * x_scale and weight * weight_scale. bias is (N,), residual (B, L, N); gate has the shapes
that the norm ops accept: (N,), (1, N), (1, 1, N), (B, N), (B, 1, N), (B, L, N) or (B or 1, F, 1, N).
K and N are multiples of 8 (K of 16 for e4m3). activation is "none", "silu", "gelu" or
"gelu_tanh". Sums are fp32; out is rounded once. Streams and devices are those of the package's
other ops.
"""
from __future__ import annotations

from typing import Optional

import torch

from . import _block_abi
from .api import _check_tensor, _operand
from .norm_quant import _out, _rows

_ACTIVATIONS = {"none": 0, "silu": 1, "gelu": 2, "gelu_tanh": 3}


def linear_gate_residual(x: torch.Tensor, weight: torch.Tensor, bias: Optional[torch.Tensor] = None,
                         gate: Optional[torch.Tensor] = None, residual: Optional[torch.Tensor] = None, *,
                         activation: str = "none", x_scale: Optional[torch.Tensor] = None,
                         weight_scale: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                         stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """residual + gate * activation(x @ weight.T + bias). `out` may be residual itself."""
    if not isinstance(x, torch.Tensor) or x.dim() != 3:
        raise ValueError("x must be a (B, L, K) tensor")
    if x.dtype not in (torch.bfloat16, torch.float16, torch.float8_e4m3fn):
        raise TypeError(f"x must be bfloat16, float16 or float8_e4m3fn, got {x.dtype}")
    if not x.is_cuda:
        raise ValueError("x must be a CUDA tensor")
    device = x.device
    B, L, K = x.shape
    _check_tensor(x, "x", device, x.dtype)
    _check_tensor(weight, "weight", device, x.dtype)
    if weight.dim() != 2 or weight.shape[1] != K:
        raise ValueError(f"weight must be an (N, {K}) matrix, got {tuple(weight.shape)}")
    N = weight.shape[0]
    if activation not in _ACTIVATIONS:
        raise ValueError(f"activation must be one of {tuple(_ACTIVATIONS)}, got {activation!r}")
    fp8 = x.dtype == torch.float8_e4m3fn
    dtype = torch.bfloat16 if fp8 else x.dtype
    a = _block_abi.lg_args(B=B, L=L, x=_rows(x, B, L), weight=weight.data_ptr(), weight_stride=weight.stride(0))
    if fp8 != (x_scale is not None) or fp8 != (weight_scale is not None):
        raise ValueError("x_scale and weight_scale are given with e4m3, and only then")
    if fp8:
        for t, name, shape in ((x_scale, "x_scale", (B, L)), (weight_scale, "weight_scale", (N,))):
            _check_tensor(t, name, device, torch.float32)
            if tuple(t.shape) != shape or not t.is_contiguous():
                raise ValueError(f"{name} must be a contiguous {shape} tensor")
        a.x_scale, a.weight_scale = x_scale.data_ptr(), weight_scale.data_ptr()
    if bias is not None:
        _check_tensor(bias, "bias", device, dtype)
        if bias.numel() != N or not bias.is_contiguous():
            raise ValueError(f"bias must be a contiguous ({N},) vector")
        a.bias = bias.data_ptr()
    if gate is not None:
        a.gate, F = _operand(gate, "gate", B, L, N, device, dtype)
        if F:
            a.tokens_per_frame = L // F
    if residual is not None:
        _check_tensor(residual, "residual", device, dtype)
        if tuple(residual.shape) != (B, L, N):
            raise ValueError(f"residual must be ({B}, {L}, {N}), got {tuple(residual.shape)}")
        a.residual = _rows(residual, B, L)
    if out is None:
        out = torch.empty((B, L, N), dtype=dtype, device=device)
    else:
        _check_tensor(_out(out, "out", (B, L, N), dtype, device), "out", device, dtype)
    a.out, (a.out_stride_b, a.out_stride_l) = out.data_ptr(), out.stride()[:2]
    key = (x.dtype, K, N, activation, bias is not None, gate is not None, residual is not None)
    h = _block_abi.handle("linear_gate", key, lambda: _block_abi.lg_config(
        _block_abi.DTYPE_CODES[x.dtype], K, N, _ACTIVATIONS[activation], int(bias is not None),
        int(gate is not None), int(residual is not None)))
    _block_abi.launch("linear_gate", h, a, device, stream)
    return out
