"""Few rows times 4-bit weights with group scales: the product of a decoding step, dense or per expert.

``matmul`` checks shapes and types, makes the output and hands pointers to ``pgemm_w4_run``; it enqueues on torch's
current stream and returns without waiting.
"""
from __future__ import annotations

import torch

from . import PGEMM_BF16, PGEMM_F16, PGEMM_W4_E2M1, PGEMM_W4_INT4, pgemm_w4_run, thread_handle
from .moe import _on_device, _records, _rows

_DTYPES = {torch.float16: PGEMM_F16, torch.bfloat16: PGEMM_BF16}
_FORMATS = {"int4": PGEMM_W4_INT4, "e2m1": PGEMM_W4_E2M1}


def matmul(x, q, scales, zeros=None, *, group: int, fmt: str = "int4", offsets=None):
    """y [M, N] = x [M, K] times the transposed 4-bit weights.

    q uint8 [N, ceil(K/2)], code k of a row in byte k // 2, the even one in the low nibble; scales of x's type
    [N, ceil(K/group)], group 32, 64 or 128. fmt "int4": (code - zero) * scale, zeros uint8 like scales (their low
    four bits), or None for 8; fmt "e2m1": the OCP 4-bit float times scale. With offsets int32 [E+1] on the device
    q, scales and zeros have a leading E, and matrix e takes x's rows offsets[e]..offsets[e+1]-1; other rows give
    zeros. For serving: it records no gradient, and refuses an x that wants one.
    """
    if _records(x):
        raise ValueError("w4.matmul has no gradient: call it under torch.no_grad() or on a detached x")
    x, ldx = _rows(x, "x")
    M, K = x.shape
    if fmt not in _FORMATS:
        raise ValueError(f"fmt {fmt!r} is not one of {sorted(_FORMATS)}")
    if group not in (32, 64, 128):
        raise ValueError(f"group {group} is not 32, 64 or 128")
    if q.dtype != torch.uint8:
        raise TypeError(f"q is {q.dtype}, not uint8")
    if scales.dtype != x.dtype:
        raise TypeError(f"scales are {scales.dtype}, x {x.dtype}")
    lead = 1 if offsets is None else 2
    if q.dim() != lead + 1 or q.shape[-1] != (K + 1) // 2:
        raise ValueError(f"q has shape {tuple(q.shape)} for K = {K}{'' if offsets is None else ' and offsets'}")
    N = q.shape[-2]
    want = tuple(q.shape[:-1]) + (-(-K // group),)
    if tuple(scales.shape) != want:
        raise ValueError(f"scales have shape {tuple(scales.shape)}, not {want}")
    tensors = [x, q, scales]
    if zeros is not None:
        if fmt != "int4":
            raise ValueError("e2m1 weights have no zero points")
        if zeros.dtype != torch.uint8:
            raise TypeError(f"zeros are {zeros.dtype}, not uint8")
        if tuple(zeros.shape) != want:
            raise ValueError(f"zeros have shape {tuple(zeros.shape)}, not {want}")
        zeros = zeros.contiguous()
        tensors.append(zeros)
    E = 1
    if offsets is not None:
        E = q.shape[0]
        if offsets.dtype != torch.int32 or tuple(offsets.shape) != (E + 1,):
            raise ValueError(f"offsets must be int32 of shape ({E + 1},)")
        if E < 1:
            raise ValueError("q holds no expert")
        offsets = offsets.contiguous()
        tensors.append(offsets)
    dev = _on_device("w4.matmul", *tensors)
    q, scales = q.contiguous(), scales.contiguous()
    y = torch.empty((M, N), dtype=x.dtype, device=dev)
    pgemm_w4_run(thread_handle(dev), x, ldx, q, scales, zeros, offsets, y, M, N, K, E, group, _FORMATS[fmt], _DTYPES[x.dtype])
    return y
