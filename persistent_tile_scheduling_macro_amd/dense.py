"""The linear layer: rows times one matrix, with bias, activation, gate and residual in the product's epilogue.

    y = dense.matmul(x, w, bias, residual, act="gelu")            # gelu(x @ w.T + bias) + residual
    h = dense.matmul(x, w_gate_up, act="silu", gated=True)        # silu(x @ gate.T) * (x @ up.T), one product

Every step runs in the HIP kernels behind the C ABI (``pgemm_dense_*``); the binding checks shapes and types, makes the
outputs and hands over pointers. The calls enqueue on torch's current stream and return without waiting. Operands are
fp16 or bf16, sums and activations fp32, each output rounded once.

``matmul`` is differentiable in x, w, bias and residual; ``matmul_backward`` is its gradient as a function of its own,
which is what to capture into a HIP graph. Errors are those of ``moe``: ValueError for shapes, TypeError for types,
PgemmError for what the library refuses, NotImplementedError for a forward-mode tangent. A tensor whose rows are not
contiguous is copied first, on every call: of a matrix that is a transposed view, pass what it is a view of with the other
layout.
"""
from __future__ import annotations

import torch
from torch.autograd.function import once_differentiable

from . import PGEMM_ACT_GELU, PGEMM_ACT_GELU_TANH, PGEMM_ACT_NONE, PGEMM_ACT_RELU, PGEMM_ACT_SILU, _ops

_ACTS = {"none": PGEMM_ACT_NONE, "relu": PGEMM_ACT_RELU, "gelu": PGEMM_ACT_GELU, "gelu_tanh": PGEMM_ACT_GELU_TANH,
         "silu": PGEMM_ACT_SILU}


def _act(act: str) -> int:
    if act not in _ACTS:
        raise ValueError(f"act {act!r} is not one of {sorted(_ACTS)}")
    return _ACTS[act]


def _nk(layout: str) -> bool:
    if layout not in ("kn", "nk"):
        raise ValueError(f"layout {layout!r} is not 'kn' or 'nk'")
    return layout == "nk"


def matmul(x, w, bias=None, residual=None, *, act: str = "none", gated: bool = False, layout: str = "nk",
           preactivation: bool = False):
    """y [M, N] = act(z) + residual with z = x times w plus bias; gated: act(z[:, :N]) * z[:, N:] + residual.

    x [M, K]; w [C, K] (layout "nk") or [K, C] ("kn"); bias [C]; residual [M, N]; C = N, or 2N where gated, the gate's
    columns first. act is "none", "relu", "gelu" (with the error function), "gelu_tanh" or "silu". With
    preactivation=True it returns (y, z), z [M, C] being what ``matmul_backward`` reads (None where it needs none; an fp16 z
    beyond 65504 is stored as that); it records no gradient, and refuses arguments that want one: call it under
    ``torch.no_grad()`` or on detached tensors.
    """
    act, nk = _act(act), _nk(layout)
    wants = torch.is_grad_enabled() and any(t is not None and t.requires_grad for t in (x, w, bias, residual))
    if preactivation:
        if wants:
            raise ValueError("dense.matmul with preactivation=True records no gradient: call it under torch.no_grad() or on "
                             "detached tensors")
        return _ops.dense(x, w, bias, residual, act, gated, nk, True)
    if wants:
        return _Dense.apply(x, w, bias, residual, act, gated, nk)
    return _ops.dense(x, w, bias, residual, act, gated, nk, False)[0]


def matmul_backward(dy, x, w, z=None, *, act: str = "none", gated: bool = False, layout: str = "nk", need_dx: bool = True,
                    need_dw: bool = True, need_dbias: bool = False):
    """(dx [M, K], dw like w, dbias [C]) from the gradient of y [M, N]; None in the place of one that is not needed.

    z: the pre-activations that ``matmul(..., preactivation=True)`` returned. The gradient of the residual is dy.
    """
    return _ops.dense_backward(dy, x, w, z, _act(act), gated, _nk(layout), need_dx, need_dw, need_dbias)


class _Dense(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, w, bias, residual, act, gated, nk):
        y, z = _ops.dense(x, w, bias, residual, act, gated, nk, True)
        ctx.save_for_backward(x, w, *(() if z is None else (z,)))
        ctx.how = act, gated, nk
        return y

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        x, w, *z = ctx.saved_tensors
        need_x, need_w, need_bias, need_residual = ctx.needs_input_grad[:4]
        grads = _ops.dense_backward(dy, x, w, z[0] if z else None, *ctx.how, need_x, need_w, need_bias)
        return *grads, dy if need_residual else None, None, None, None
