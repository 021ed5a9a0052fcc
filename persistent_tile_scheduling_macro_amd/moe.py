"""Mixture-of-experts operators: token rows to their experts, the experts' products, and back.

A layer is four kinds of call::

    ids, weights = moe.route(logits, k)                        # each token's experts
    xs, plan = moe.dispatch(x, ids, E)                         # rows sorted by expert
    ys = moe.grouped_matmul(xs, w, plan.offsets, layout="nk")  # each row times its expert's matrix
    out = moe.combine(ys, weights, plan)                       # the token's rows, weighted and summed

and for the few tokens of a decoding batch the last three are one::

    out = moe.layer(x, ids, weights, w_in, w_out, act="silu", gated=True)

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

from . import PGEMM_SCORE_SIGMOID, PGEMM_SCORE_SOFTMAX, _ops
from .dense import _act


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


# ------------------------------------------------------------------ router
_SCORES = {"softmax": PGEMM_SCORE_SOFTMAX, "sigmoid": PGEMM_SCORE_SIGMOID}


def _score(score: str) -> int:
    if score not in _SCORES:
        raise ValueError(f"score {score!r} is not one of {sorted(_SCORES)}")
    return _SCORES[score]


def route(logits, k: int, *, score: str = "softmax", normalize: bool = True):
    """Each token's k experts and their weights: (ids int32 [T, k], weights float32 [T, k]).

    logits [T, E], float32, bf16 or fp16. The largest are chosen, largest first, the first of equal ones first; -inf and
    NaN never, and a token with fewer than k others gets ids of -1 with weights of 0 in the places left, which
    ``dispatch`` drops. The weights are the chosen scores, the softmax over all experts or each logit's sigmoid; with
    normalize they are divided by their sum. Differentiable in logits, through the weights.
    """
    if _records(logits):
        return _Route.apply(logits, k, _score(score), bool(normalize))
    return _ops.route(logits, k, _score(score), bool(normalize))


def route_backward(dweights, logits, ids, weights, *, score: str = "softmax", normalize: bool = True):
    """Gradient of logits [T, E] from the gradient of the weights [T, k], with what ``route`` took and returned."""
    return _ops.route_backward(dweights, logits, ids, weights, _score(score), bool(normalize))


class _Route(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, k, score, normalize):
        ids, weights = _ops.route(logits, k, score, normalize)
        ctx.save_for_backward(logits, ids, weights)
        ctx.how = score, normalize
        ctx.mark_non_differentiable(ids)
        return ids, weights

    @staticmethod
    @once_differentiable
    def backward(ctx, _, dweights):
        return _ops.route_backward(dweights, *ctx.saved_tensors, *ctx.how), None, None, None


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


# --------------------------------------------------- a whole layer of few tokens
def layer(x, ids, weights, w_in, w_out, *, act: str = "silu", gated: bool = True):
    """out[t] = sum over j of weights[t, j] * (a(x[t]) @ w_out[e].T) with e = ids[t, j], in two launches for each 64 tokens.

    x [T, H]; ids int32 or int64 [T, k] (outside [0, E): dropped); weights float32 [T, k]; a(x) = act(x @ w_in[e].T) with
    w_in [E, I, H], or, gated, w_in [E, 2I, H] and act of the first I columns times the others; w_out [E, H, I]; act as
    in ``dense.matmul``. Each expert that a token names is read once for 64 tokens (up to four times where most of them
    name it), so it is for the few tokens of a decoding batch. It takes up to 4096, but more than 64 read the matrices
    again: with 8 of 64 experts of 2048 x 1024 ``dispatch``, ``grouped_matmul`` and ``combine`` with torch's operations
    between them are as fast at 64 tokens (192 us) and take 222 us for 128, where this takes 384. Matrices that are not
    contiguous are copied whole on every call. The ids of all tokens fix the order of the sums: a batch's results are
    always the same, but a token's last bits may depend on the tokens beside it. For serving: it records no gradient, and
    refuses arguments that want one.
    """
    if torch.is_grad_enabled() and any(t.requires_grad for t in (x, weights, w_in, w_out)):
        raise ValueError("moe.layer has no gradient: call it under torch.no_grad() or on detached tensors")
    return _ops.layer(x, ids, weights, w_in, w_out, _act(act), gated)
