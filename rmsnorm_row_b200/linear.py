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
K and N are multiples of 8 (K of 16 for e4m3). Rows of x and
(N,) vectors start at 16 bytes; beyond four tokens x has a row of its own for each (no expanded x).
Many short batches that lie apart (x[:, :2] of a longer tensor) are slow, up to 128 / L times the
same tokens in one piece: call .contiguous() on them. activation is "none", "silu", "gelu" or
"gelu_tanh". Sums are fp32; out is rounded once. Streams and devices are those of the package's
other ops. The function is not recorded by autograd: its result requires no gradient, whatever its
inputs do.

The matrix kernel bounds its internal waits. A call in which one ran out (ten seconds) leaves its
output incomplete: the next call raises FusedNormError, and ``linear_gate_timeouts`` counts it.
"""
from __future__ import annotations

import ctypes
from typing import Optional

import torch

from . import _block_abi
from ._block_abi import binding


def linear_gate_residual(x: torch.Tensor, weight: torch.Tensor, bias: Optional[torch.Tensor] = None,
                         gate: Optional[torch.Tensor] = None, residual: Optional[torch.Tensor] = None, *,
                         activation: str = "none", x_scale: Optional[torch.Tensor] = None,
                         weight_scale: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                         stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """residual + gate * activation(x @ weight.T + bias). `out` may be residual itself."""
    return binding().linear_gate(x, weight, bias, gate, residual, activation, x_scale, weight_scale, out, stream)


def linear_gate_timeouts(device: Optional[torch.device] = None) -> int:
    """How many CTAs of linear_gate_residual on `device` (default: the current one) have given up a wait
    since the library was loaded. Synchronises with the device's default stream."""
    n = ctypes.c_int()
    with torch.cuda.device(device):
        _block_abi.check(_block_abi.load().linear_gate_timeouts(ctypes.byref(n)), "linear_gate_timeouts")
    return n.value
