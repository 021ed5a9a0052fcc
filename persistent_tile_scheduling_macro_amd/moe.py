"""Mixture-of-experts operators: token rows to their experts, the experts' products, and back.

A layer is three kinds of call::

    xs, plan = moe.dispatch(x, ids, E)                         # rows sorted by expert
    ys = moe.grouped_matmul(xs, w, plan.offsets, layout="nk")  # each row times its expert's matrix
    out = moe.combine(ys, weights, plan)                       # the token's rows, weighted and summed

Every step runs in the HIP kernels behind the C ABI (``pgemm_moe_*``, ``pgemm_grouped_*``); the binding checks shapes
and types, makes the outputs and hands over pointers. The calls enqueue on torch's current stream and return without
waiting. Rows are fp16 or bf16, sums fp32 rounded once.

The functions are differentiable: where torch records gradients they enter its graph, and each gradient is
also a function of its own (``*_backward``), which is what to capture into a HIP graph. Tensors of the wrong shape
raise ValueError, of the wrong type TypeError, a refusal of the library raises PgemmError, a tensor that carries a
forward-mode tangent NotImplementedError. A tensor whose rows are not contiguous is copied first.
"""
from __future__ import annotations

import torch
from torch.autograd.function import once_differentiable

from . import _ops


class RoutePlan:
    """Where the T*k slots of a batch went: what ``dispatch`` returns and the other steps read.

    offsets int32 [E+1], order int32 [T*k], pos int32 [T*k] (see pgemm.h), and k, the slots of a token. A slot is taken
    out afterwards by setting its pos to -1 (its row stays where it is, without a share and with a gradient of zeros).
    """

    __slots__ = ("offsets", "order", "pos", "k")

    def __init__(self, offsets, order, pos, k: int):
        self.offsets, self.order, self.pos, self.k = offsets, order, pos, int(k)


def _records(a, b=None) -> bool:
    return (a.requires_grad or (b is not None and b.requires_grad)) and torch.is_grad_enabled()


# ---------------------------------------------------------------- dispatch
def dispatch(x, ids, num_experts: int):
    """Sort the slots of x's tokens by expert: (xs, plan).

    x [T, H]; ids int32 or int64 [T, k], the experts of each token (an id outside [0, num_experts) drops its slot).
    xs [T*k, H] holds x's rows in the plan's order, zeros behind the last kept one. Differentiable in x.
    """
    call = _Dispatch.apply if _records(x) else _ops.dispatch
    xs, offsets, order, pos = call(x, ids, num_experts)
    return xs, RoutePlan(offsets, order, pos, ids.shape[1])


def dispatch_backward(dxs, plan: RoutePlan):
    """Gradient of x [T, H] from the gradient of xs [T*k, H]: the token's kept rows, summed in fp32."""
    return _ops.dispatch_backward(dxs, plan.offsets, plan.order, plan.pos, plan.k)


class _Dispatch(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, ids, num_experts):
        xs, *plan = _ops.dispatch(x, ids, num_experts)
        ctx.save_for_backward(*plan)
        ctx.k = ids.shape[1]
        ctx.mark_non_differentiable(*plan)
        return xs, *plan

    @staticmethod
    @once_differentiable
    def backward(ctx, dxs, *_):
        return _ops.dispatch_backward(dxs, *ctx.saved_tensors, ctx.k), None, None


# ----------------------------------------------------------------- combine
def combine(ys, weights, plan: RoutePlan):
    """out[t] = sum over the token's kept slots of weights[t, j] * ys[its sorted row].

    ys [T*k, H]; weights float32 [T, k]; out [T, H] in ys's type. Differentiable in ys and weights.
    """
    call = _Combine.apply if _records(ys, weights) else _ops.combine
    return call(ys, weights, plan.offsets, plan.order, plan.pos, plan.k)


def combine_backward(dout, ys, weights, plan: RoutePlan):
    """(dys [T*k, H], dweights float32 [T, k]) from the gradient of out [T, H]."""
    return _ops.combine_backward(dout, ys, weights, plan.offsets, plan.order, plan.pos, plan.k)


class _Combine(torch.autograd.Function):
    @staticmethod
    def forward(ctx, ys, weights, offsets, order, pos, k):
        ctx.save_for_backward(ys, weights, offsets, order, pos)
        ctx.k = k
        return _ops.combine(ys, weights, offsets, order, pos, k)

    @staticmethod
    @once_differentiable
    def backward(ctx, dout):
        return *_ops.combine_backward(dout, *ctx.saved_tensors, ctx.k), None, None, None, None


# -------------------------------------------------------- the experts' products
def _nk(layout: str) -> bool:
    if layout not in ("kn", "nk"):
        raise ValueError(f"layout {layout!r} is not 'kn' or 'nk'")
    return layout == "nk"


def grouped_matmul(x, w, offsets, *, layout: str = "nk"):
    """y[r] = x[r] @ w[e] for the rows r = offsets[e] .. offsets[e+1]-1 of every expert e, zeros in other rows.

    x [R, K]; w [E, K, N] (layout "kn") or [E, N, K] ("nk"); offsets int32 [E+1] on the device, as in a plan (they are
    never read by the host); y [R, N]. Differentiable in x and w.
    """
    return (_Grouped.apply if _records(x, w) else _ops.grouped)(x, w, offsets, _nk(layout))


def grouped_matmul_backward(dy, x, w, offsets, *, layout: str = "nk", need_dx: bool = True, need_dw: bool = True):
    """(dx [R, K], dw like w) from the gradient of y [R, N]; None in the place of one that is not needed."""
    return _ops.grouped_backward(dy, x, w, offsets, _nk(layout), need_dx, need_dw)


class _Grouped(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, w, offsets, nk):
        ctx.save_for_backward(x, w, offsets)
        ctx.nk = nk
        return _ops.grouped(x, w, offsets, nk)

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        return *_ops.grouped_backward(dy, *ctx.saved_tensors, ctx.nk, *ctx.needs_input_grad[:2]), None, None
