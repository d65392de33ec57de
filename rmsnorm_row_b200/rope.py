"""RMS norm of q or k with rotary positions over several axes, and its gradient
(include/block_ops.h, rope_norm).

    rope_norm(x, positions, sections, weight=None) -> y
    rope_norm_backward(grad, x, positions, sections, weight=None) -> (dx, dweight)

x is (B, L, H, hd), bf16 or fp16, with contiguous channels (a slice of a packed qkv
projection will do); positions is (L, axes), or (B, L, axes) or (1, L, axes), int32 or int64;
sections gives the pairs of channels that follow each axis, e.g. (22, 21, 21) of a head of 128
for (time, height, width). Channels beyond 2 * sum(sections) pass through the rotation.

norm is "all" (over the H * hd channels of a token, weight of H * hd), "head" (weight of hd)
or "none"; weight is optional, of x's dtype or fp32. pairing is "interleaved" (channels 2i and
2i + 1) or "half" (i and i + sum(sections)). Each section has frequencies theta^(-i / pairs of
the section), or, with shared_frequencies, pair i of all has theta^(-i / sum(sections)).

The functions are not recorded by autograd: a training step calls rope_norm_backward with the
forward's inputs. Streams and devices are those of the package's other ops.
"""
from __future__ import annotations

from typing import Optional, Sequence, Tuple

import torch

from . import _block_abi

_NORMS = {"none": 0, "head": 1, "all": 2}
_PAIRINGS = {"interleaved": 0, "half": 1}


def _heads(t: torch.Tensor, name: str, like: Optional[torch.Tensor] = None) -> "_block_abi.rn_rows":
    """The rows of a (B, L, H, hd) tensor, of `like`'s shape, dtype and device where given."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dim() != 4:
        raise ValueError(f"{name} must be a (B, L, H, hd) tensor")
    if t.dtype not in (torch.bfloat16, torch.float16):
        raise TypeError(f"{name} must be bfloat16 or float16, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if like is not None and (t.shape != like.shape or t.dtype != like.dtype or t.device != like.device):
        raise ValueError(f"{name} must be a {like.dtype} tensor of shape {tuple(like.shape)} on {like.device}")
    B, L, H, hd = t.shape
    sb, sl, sh, sc = t.stride()
    if sc != 1 and hd > 1:
        raise ValueError(f"{name} needs contiguous channels")
    return _block_abi.rn_rows(t.data_ptr(), sb if B > 1 else 0, sl if L > 1 else 0, sh if H > 1 else 0)


def _prepare(x, positions, sections, weight, theta, pairing, shared_frequencies, norm, eps):
    """(handle, positions' strides) for a call on x."""
    B, L, H, hd = x.shape
    if norm not in _NORMS:
        raise ValueError(f"norm must be one of {tuple(_NORMS)}, got {norm!r}")
    if pairing not in _PAIRINGS:
        raise ValueError(f"pairing must be one of {tuple(_PAIRINGS)}, got {pairing!r}")
    sections = tuple(int(n) for n in sections)
    axes = len(sections)
    if not 1 <= axes <= 4 or min(sections) < 1:
        raise ValueError(f"sections must be one to four positive numbers, got {sections}")
    if not isinstance(positions, torch.Tensor) or positions.dtype not in (torch.int32, torch.int64):
        raise TypeError("positions must be an int32 or int64 tensor")
    if positions.device != x.device:
        raise ValueError(f"positions is on {positions.device}, expected {x.device}")
    ok = positions.dim() in (2, 3) and tuple(positions.shape[-2:]) == (L, axes)
    if not ok or (positions.dim() == 3 and positions.shape[0] not in (1, B)):
        raise ValueError(f"positions must be ({L}, {axes}) or ({B}, {L}, {axes}), got {tuple(positions.shape)}")
    s = positions.stride()
    if axes > 1 and s[-1] != 1:
        raise ValueError("positions needs a contiguous last dimension")
    pos = (s[0] if positions.dim() == 3 and positions.shape[0] > 1 else 0, s[-2] if L > 1 else 0)
    fp32 = False
    if weight is not None:
        if norm == "none":
            raise ValueError("weight needs a norm")
        if not isinstance(weight, torch.Tensor) or weight.dtype not in (x.dtype, torch.float32):
            raise TypeError(f"weight must be a {x.dtype} or float32 tensor")
        n = H * hd if norm == "all" else hd
        if weight.device != x.device or weight.numel() != n or not weight.is_contiguous():
            raise ValueError(f"weight must be a contiguous ({n},) vector on {x.device}")
        fp32 = weight.dtype == torch.float32
    key = (x.dtype, H, hd, sections, norm, weight is not None, fp32, pairing, bool(shared_frequencies),
           positions.dtype, float(theta), float(eps))

    def config():
        return _block_abi.rn_config(
            _block_abi.DTYPE_CODES[x.dtype], H, hd, axes, (_block_abi.c_int4)(*sections), _NORMS[norm],
            int(weight is not None), int(fp32), _PAIRINGS[pairing], int(bool(shared_frequencies)),
            int(positions.dtype == torch.int64), float(theta), float(eps))

    return _block_abi.handle("rope_norm", key, config), pos


def rope_norm(x: torch.Tensor, positions: torch.Tensor, sections: Sequence[int],
              weight: Optional[torch.Tensor] = None, *, theta: float = 10000.0, pairing: str = "interleaved",
              shared_frequencies: bool = False, norm: str = "all", eps: float = 1e-6,
              out: Optional[torch.Tensor] = None, stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """x normed, weighted and turned by its positions. `out` may be x itself."""
    rows = _heads(x, "x")
    h, (psb, psl) = _prepare(x, positions, sections, weight, theta, pairing, shared_frequencies, norm, eps)
    y = torch.empty(x.shape, dtype=x.dtype, device=x.device) if out is None else out
    a = _block_abi.rn_args(x.shape[0], x.shape[1], rows, positions.data_ptr(), psb, psl,
                           None if weight is None else weight.data_ptr(), _heads(y, "out", x))
    _block_abi.launch("rope_norm", h, a, x.device, stream)
    return y


def rope_norm_backward(grad: torch.Tensor, x: torch.Tensor, positions: torch.Tensor, sections: Sequence[int],
                       weight: Optional[torch.Tensor] = None, *, theta: float = 10000.0,
                       pairing: str = "interleaved", shared_frequencies: bool = False, norm: str = "all",
                       eps: float = 1e-6, out: Optional[torch.Tensor] = None,
                       stream: Optional[torch.cuda.Stream] = None) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """(dx, dweight) of rope_norm(x, ...) for the gradient of its output: dx like x, dweight fp32
    (None without a weight), the same in every run. `out` is dx's tensor and may be grad or x."""
    rows = _heads(x, "x")
    dy = _heads(grad, "grad", x)
    h, (psb, psl) = _prepare(x, positions, sections, weight, theta, pairing, shared_frequencies, norm, eps)
    dx = torch.empty(x.shape, dtype=x.dtype, device=x.device) if out is None else out
    dw = work = None
    B, L = x.shape[:2]
    if weight is not None:
        dw = torch.empty(weight.shape, dtype=torch.float32, device=x.device)
        work = torch.empty(_block_abi.rope_norm_workspace(h, B, L), dtype=torch.uint8, device=x.device)
        if stream is not None:  # dropped here, in use on that stream
            work.record_stream(stream)
    if norm == "none":
        rows = _block_abi.rn_rows(None, 0, 0, 0)
    a = _block_abi.rn_backward_args(
        B, L, dy, rows, positions.data_ptr(), psb, psl, None if weight is None else weight.data_ptr(),
        _heads(dx, "out", x), None if dw is None else dw.data_ptr(),
        None if work is None else work.data_ptr() or None, 0 if work is None else work.numel())
    _block_abi.launch("rope_norm", h, a, x.device, stream, call="backward_launch")
    return dx, dw
