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

The functions are not recorded by autograd (their results require no gradient): a training step
calls rope_norm_backward with the forward's inputs. Streams and devices are those of the package's other ops.
"""
from __future__ import annotations

from typing import Optional, Sequence, Tuple

import torch

from ._block_abi import binding


def rope_norm(x: torch.Tensor, positions: torch.Tensor, sections: Sequence[int],
              weight: Optional[torch.Tensor] = None, *, theta: float = 10000.0, pairing: str = "interleaved",
              shared_frequencies: bool = False, norm: str = "all", eps: float = 1e-6,
              out: Optional[torch.Tensor] = None, stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """x normed, weighted and turned by its positions. `out` may be x itself."""
    return binding().rope_norm(x, positions, sections, weight, theta, pairing, shared_frequencies, norm, eps, out, stream)


def rope_norm_backward(grad: torch.Tensor, x: torch.Tensor, positions: torch.Tensor, sections: Sequence[int],
                       weight: Optional[torch.Tensor] = None, *, theta: float = 10000.0,
                       pairing: str = "interleaved", shared_frequencies: bool = False, norm: str = "all",
                       eps: float = 1e-6, out: Optional[torch.Tensor] = None,
                       stream: Optional[torch.cuda.Stream] = None) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """(dx, dweight) of rope_norm(x, ...) for the gradient of its output: dx like x, dweight fp32
    (None without a weight), the same in every run. `out` is dx's tensor and may be grad or x."""
    return binding().rope_norm_backward(grad, x, positions, sections, weight, theta, pairing, shared_frequencies, norm,
                                        eps, out, stream)
