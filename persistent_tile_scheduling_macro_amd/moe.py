"""Mixture-of-experts operators: token rows to their experts, the experts' products, and back.

A layer is four calls::

    xs, plan = moe.dispatch(x, ids, E)                         # rows sorted by expert
    ys = moe.grouped_matmul(xs, w, plan.offsets, layout="nk")  # each row times its expert's matrix
    out = moe.combine(ys, weights, plan)                       # the token's rows, weighted and summed

Every step runs in the HIP kernels behind the C ABI (``pgemm_moe_*``, ``pgemm_grouped_*``); the functions here check
shapes and types, make the outputs and hand over pointers. They enqueue on torch's current stream and return without
waiting. Rows are fp16 or bf16, sums fp32 rounded once.

The functions are differentiable: where torch records gradients they enter its graph, and each gradient is
also a function of its own (``*_backward``). Tensors of the wrong shape or type raise ValueError or TypeError, a
refusal of the library PgemmError. A tensor whose rows are not contiguous is copied first.
"""
from __future__ import annotations

import torch
from torch.autograd.function import once_differentiable

from . import (PGEMM_B_KN, PGEMM_B_NK, PGEMM_BF16, PGEMM_F16, PGEMM_IDS_I32, PGEMM_IDS_I64, pgemm_grouped_run,
               pgemm_grouped_weight_grad, pgemm_moe_combine, pgemm_moe_combine_backward, pgemm_moe_dispatch,
               pgemm_moe_dispatch_backward, pgemm_moe_dispatch_workspace, thread_handle)

_DTYPES = {torch.float16: PGEMM_F16, torch.bfloat16: PGEMM_BF16}
_IDS = {torch.int32: PGEMM_IDS_I32, torch.int64: PGEMM_IDS_I64}


class RoutePlan:
    """Where the T*k slots of a batch went: what ``dispatch`` returns and the other steps read.

    offsets int32 [E+1], order int32 [T*k], pos int32 [T*k] (see pgemm.h), and k, the slots of a token.
    """

    __slots__ = ("offsets", "order", "pos", "k")

    def __init__(self, offsets, order, pos, k: int):
        self.offsets, self.order, self.pos, self.k = offsets, order, pos, int(k)

    def _sizes(self, name: str):
        """(T, n) after checking the plan's tensors."""
        n = self.pos.numel()
        for what, t in (("offsets", self.offsets), ("order", self.order), ("pos", self.pos)):
            if t.dtype != torch.int32 or t.dim() != 1 or not t.is_contiguous():
                raise ValueError(f"{name}: plan.{what} must be a contiguous int32 vector")
        if self.k < 1 or n % self.k or self.order.numel() != n or self.offsets.numel() < 2:
            raise ValueError(f"{name}: the plan's sizes do not belong together")
        return n // self.k, n


def _rows(t, name: str, shape=None):
    """A 2-D fp16/bf16 tensor whose rows are contiguous, and its row stride in elements."""
    if t.dtype not in _DTYPES:
        raise TypeError(f"{name} is {t.dtype}, not float16 or bfloat16")
    if t.dim() != 2:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, not two dimensions")
    if shape is not None and tuple(t.shape) != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, not {shape}")
    if t.stride(1) != 1 and t.shape[1] > 1:
        t = t.contiguous()
    return t, t.stride(0)


def _on_device(name: str, *tensors):
    dev = tensors[0].device
    for t in tensors:
        if not t.is_cuda:
            raise ValueError(f"{name}: every tensor must be on the GPU")
        if t.device != dev:
            raise ValueError(f"{name}: tensors on {dev} and {t.device}")
    return dev


def _records(*tensors) -> bool:
    return torch.is_grad_enabled() and any(t.requires_grad for t in tensors)


# ---------------------------------------------------------------- dispatch
def dispatch(x, ids, num_experts: int):
    """Sort the slots of x's tokens by expert: (xs, plan).

    x [T, H]; ids int32 or int64 [T, k], the experts of each token (an id outside [0, num_experts) drops its slot).
    xs [T*k, H] holds x's rows in the plan's order, zeros behind the last kept one. Differentiable in x.
    """
    if _records(x):
        xs, offsets, order, pos = _Dispatch.apply(x, ids, num_experts)
        return xs, RoutePlan(offsets, order, pos, ids.shape[1])
    return _dispatch(x, ids, num_experts)


def _dispatch(x, ids, num_experts):
    x, ldx = _rows(x, "x")
    T, H = x.shape
    if ids.dtype not in _IDS:
        raise TypeError(f"ids are {ids.dtype}, not int32 or int64")
    if ids.dim() != 2 or ids.shape[0] != T or ids.shape[1] < 1:
        raise ValueError(f"ids have shape {tuple(ids.shape)}, not ({T}, k)")
    E, k = int(num_experts), ids.shape[1]
    if E < 1:
        raise ValueError(f"num_experts is {num_experts}")
    dev = _on_device("dispatch", x, ids)
    ids = ids.contiguous()
    n = T * k
    work_bytes = pgemm_moe_dispatch_workspace(T, k, E)
    h = thread_handle(dev)
    offsets = torch.empty(E + 1, dtype=torch.int32, device=dev)
    order = torch.empty(n, dtype=torch.int32, device=dev)
    pos = torch.empty(n, dtype=torch.int32, device=dev)
    xs = torch.empty((n, H), dtype=x.dtype, device=dev)
    work = torch.empty(work_bytes, dtype=torch.uint8, device=dev) if work_bytes else None
    pgemm_moe_dispatch(h, x, ldx, ids, _IDS[ids.dtype], T, k, E, H, _DTYPES[x.dtype], offsets, order, pos, xs, work,
                       work_bytes)
    return xs, RoutePlan(offsets, order, pos, k)


def dispatch_backward(dxs, plan: RoutePlan):
    """Gradient of x [T, H] from the gradient of xs [T*k, H]: the token's kept rows, summed in fp32."""
    T, n = plan._sizes("dispatch_backward")
    dxs, ld = _rows(dxs, "dxs")
    if dxs.shape[0] != n:
        raise ValueError(f"dxs has {dxs.shape[0]} rows, the plan {n}")
    dev = _on_device("dispatch_backward", dxs, plan.pos)
    H = dxs.shape[1]
    h = thread_handle(dev)
    dx = torch.empty((T, H), dtype=dxs.dtype, device=dev)
    pgemm_moe_dispatch_backward(h, dxs, ld, plan.pos, T, plan.k, H, _DTYPES[dxs.dtype], dx)
    return dx


class _Dispatch(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, ids, num_experts):
        xs, plan = _dispatch(x, ids, num_experts)
        ctx.plan = plan
        ctx.mark_non_differentiable(plan.offsets, plan.order, plan.pos)
        return xs, plan.offsets, plan.order, plan.pos

    @staticmethod
    @once_differentiable
    def backward(ctx, dxs, *_):
        return dispatch_backward(dxs, ctx.plan), None, None


# ----------------------------------------------------------------- combine
def _check_combine(name, ys, weights, plan):
    T, n = plan._sizes(name)
    ys, ld = _rows(ys, "ys")
    if ys.shape[0] != n:
        raise ValueError(f"{name}: ys has {ys.shape[0]} rows, the plan {n}")
    if weights.dtype != torch.float32:
        raise TypeError(f"{name}: weights are {weights.dtype}, not float32")
    if tuple(weights.shape) != (T, plan.k):
        raise ValueError(f"{name}: weights have shape {tuple(weights.shape)}, not {(T, plan.k)}")
    return ys, ld, weights.contiguous(), T, n


def combine(ys, weights, plan: RoutePlan):
    """out[t] = sum over the token's kept slots of weights[t, j] * ys[its sorted row].

    ys [T*k, H]; weights float32 [T, k]; out [T, H] in ys's type. Differentiable in ys and weights.
    """
    if _records(ys, weights):
        return _Combine.apply(ys, weights, plan)
    return _combine(ys, weights, plan)


def _combine(ys, weights, plan):
    ys, ld, weights, T, n = _check_combine("combine", ys, weights, plan)
    dev = _on_device("combine", ys, weights, plan.pos)
    H = ys.shape[1]
    h = thread_handle(dev)
    out = torch.empty((T, H), dtype=ys.dtype, device=dev)
    pgemm_moe_combine(h, ys, ld, weights, plan.pos, T, plan.k, H, _DTYPES[ys.dtype], out)
    return out


def combine_backward(dout, ys, weights, plan: RoutePlan):
    """(dys [T*k, H], dweights float32 [T, k]) from the gradient of out [T, H]."""
    ys, ldys, weights, T, n = _check_combine("combine_backward", ys, weights, plan)
    H = ys.shape[1]
    dout, lddout = _rows(dout, "dout", (T, H))
    if dout.dtype != ys.dtype:
        raise TypeError(f"combine_backward: dout is {dout.dtype}, ys {ys.dtype}")
    dev = _on_device("combine_backward", ys, dout, weights, plan.pos, plan.offsets)
    h = thread_handle(dev)
    dys = torch.empty((n, H), dtype=ys.dtype, device=dev)
    dw = torch.empty((T, plan.k), dtype=torch.float32, device=dev)
    pgemm_moe_combine_backward(h, dout, lddout, ys, ldys, weights, plan.offsets, plan.pos, T, plan.k,
                               plan.offsets.numel() - 1, H, _DTYPES[ys.dtype], dys, dw)
    return dys, dw


class _Combine(torch.autograd.Function):
    @staticmethod
    def forward(ctx, ys, weights, plan):
        ctx.save_for_backward(ys, weights)
        ctx.plan = plan
        return _combine(ys, weights, plan)

    @staticmethod
    @once_differentiable
    def backward(ctx, dout):
        ys, weights = ctx.saved_tensors
        dys, dw = combine_backward(dout, ys, weights, ctx.plan)
        return dys, dw, None


# -------------------------------------------------------- the experts' products
_LAYOUTS = {"kn": PGEMM_B_KN, "nk": PGEMM_B_NK}
_OTHER = {"kn": "nk", "nk": "kn"}


def _check_grouped(name, x, w, offsets, layout):
    """(x, ldx, w, offsets, K, N) after checking them."""
    x, ldx = _rows(x, "x")
    if layout not in _LAYOUTS:
        raise ValueError(f"{name}: layout {layout!r} is not one of {sorted(_LAYOUTS)}")
    if w.dtype != x.dtype:
        raise TypeError(f"{name}: w is {w.dtype}, x {x.dtype}")
    K = x.shape[1]
    if w.dim() != 3 or w.shape[0] < 1 or w.shape[1 if layout == "kn" else 2] != K:
        raise ValueError(f"{name}: w has shape {tuple(w.shape)} for rows of {K} and layout {layout!r}")
    if offsets.dtype != torch.int32 or tuple(offsets.shape) != (w.shape[0] + 1,):
        raise ValueError(f"{name}: offsets must be int32 of shape ({w.shape[0] + 1},)")
    _on_device(name, x, w, offsets)
    return x, ldx, w.contiguous(), offsets.contiguous(), K, w.shape[2 if layout == "kn" else 1]


def grouped_matmul(x, w, offsets, *, layout: str = "nk"):
    """y[r] = x[r] @ w[e] for the rows r = offsets[e] .. offsets[e+1]-1 of every expert e, zeros in other rows.

    x [R, K]; w [E, K, N] (layout "kn") or [E, N, K] ("nk"); offsets int32 [E+1] on the device, as in a plan (they are
    never read by the host); y [R, N]. Differentiable in x and w.
    """
    if _records(x, w):
        return _Grouped.apply(x, w, offsets, layout)
    return _grouped(x, w, offsets, layout)


def _grouped(x, w, offsets, layout):
    x, ldx, w, offsets, K, N = _check_grouped("grouped_matmul", x, w, offsets, layout)
    R = x.shape[0]
    y = torch.empty((R, N), dtype=x.dtype, device=x.device)
    pgemm_grouped_run(thread_handle(x.device), x, ldx, w, offsets, y, R, w.shape[0], K, N, _LAYOUTS[layout],
                      _DTYPES[x.dtype])
    return y


def _grouped_dw(dy, x, offsets, E, layout):
    a, b = (x, dy) if layout == "kn" else (dy, x)
    dw = torch.empty((E, a.shape[1], b.shape[1]), dtype=x.dtype, device=x.device)
    pgemm_grouped_weight_grad(thread_handle(x.device), a, a.stride(0), b, b.stride(0), offsets, dw, x.shape[0], E,
                              a.shape[1], b.shape[1], _DTYPES[x.dtype])
    return dw


def grouped_matmul_backward(dy, x, w, offsets, *, layout: str = "nk", need_dx: bool = True, need_dw: bool = True):
    """(dx [R, K], dw like w) from the gradient of y [R, N]; None in the place of one that is not needed."""
    x, _, w, offsets, K, N = _check_grouped("grouped_matmul_backward", x, w, offsets, layout)
    dy, _ = _rows(dy, "dy", (x.shape[0], N))
    if dy.dtype != x.dtype:
        raise TypeError(f"grouped_matmul_backward: dy is {dy.dtype}, x {x.dtype}")
    _on_device("grouped_matmul_backward", x, dy)
    dx = _grouped(dy, w, offsets, _OTHER[layout]) if need_dx else None
    dw = _grouped_dw(dy, x, offsets, w.shape[0], layout) if need_dw else None
    return dx, dw


class _Grouped(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, w, offsets, layout):
        ctx.save_for_backward(x, w, offsets)
        ctx.layout = layout
        return _grouped(x, w, offsets, layout)

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        x, w, offsets = ctx.saved_tensors
        dx, dw = grouped_matmul_backward(dy, x, w, offsets, layout=ctx.layout, need_dx=ctx.needs_input_grad[0],
                                         need_dw=ctx.needs_input_grad[1])
        return dx, dw, None, None
