"""Few rows times 4-bit weights with group scales: the product of a decoding step, dense or per expert.

``matmul`` checks shapes and types, makes the output and hands pointers to ``pgemm_w4_run``; it enqueues on torch's
current stream and returns without waiting.
"""
from __future__ import annotations

import torch

from . import PGEMM_W4_E2M1, PGEMM_W4_INT4, _ops

_FORMATS = {"int4": PGEMM_W4_INT4, "e2m1": PGEMM_W4_E2M1}


def matmul(x, q, scales, zeros=None, *, group: int, fmt: str = "int4", offsets=None):
    """y [M, N] = x [M, K] times the transposed 4-bit weights.

    q uint8 [N, ceil(K/2)], code k of a row in byte k // 2, the even one in the low nibble; scales of x's type
    [N, ceil(K/group)], group 32, 64 or 128. fmt "int4": (code - zero) * scale, zeros uint8 like scales (their low
    four bits), or None for 8; fmt "e2m1": the OCP 4-bit float times scale. With offsets int32 [E+1] on the device
    q, scales and zeros have a leading E, and matrix e takes x's rows offsets[e]..offsets[e+1]-1; other rows give
    zeros. For serving: it records no gradient, and refuses an x or scales that want one.
    """
    if (x.requires_grad or scales.requires_grad) and torch.is_grad_enabled():
        raise ValueError("w4.matmul has no gradient: call it under torch.no_grad() or on detached x and scales")
    if fmt not in _FORMATS:
        raise ValueError(f"fmt {fmt!r} is not one of {sorted(_FORMATS)}")
    return _ops.w4(x, q, scales, zeros, group, _FORMATS[fmt], offsets)
