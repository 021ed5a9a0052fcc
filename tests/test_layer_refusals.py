"""CPU: what the linear layer, the router and the routed layer of few tokens refuse, before any device work."""
import pytest
import torch
import torch.autograd.forward_ad as fwd

import persistent_tile_scheduling_macro_amd as pg
from persistent_tile_scheduling_macro_amd import dense, moe

F16, BF16, F32, I32, I64 = torch.float16, torch.bfloat16, torch.float32, torch.int32, torch.int64


def t(*shape, dtype=F16):
    return torch.zeros(shape, dtype=dtype)


def layer(x=(4, 8), ids=(4, 2), weights=(4, 2), w_in=(3, 12, 8), w_out=(3, 8, 6), dt=F16, ids_dt=I32, wt=F32, wout_dt=None, **how):
    return moe.layer(t(*x, dtype=dt), t(*ids, dtype=ids_dt), t(*weights, dtype=wt), t(*w_in, dtype=dt),
                     t(*w_out, dtype=wout_dt or dt), **how)


@pytest.mark.parametrize("error,call", [
    (TypeError, lambda: dense.matmul(t(4, 8, dtype=F32), t(6, 8, dtype=F32))),
    (TypeError, lambda: dense.matmul(t(4, 8), t(6, 8, dtype=BF16))),
    (ValueError, lambda: dense.matmul(t(4, 8, 1), t(6, 8))),
    (ValueError, lambda: dense.matmul(t(4, 8), t(6, 9))),
    (ValueError, lambda: dense.matmul(t(4, 8), t(6, 8), layout="kn")),
    (ValueError, lambda: dense.matmul(t(4, 8), t(6, 8), layout="mn")),
    (ValueError, lambda: dense.matmul(t(4, 8), t(6, 8), act="tanh")),
    (ValueError, lambda: dense.matmul(t(4, 8), t(7, 8), gated=True)),
    (ValueError, lambda: dense.matmul(t(4, 8), t(6, 8))),  # not on the GPU
    (ValueError, lambda: dense.matmul_backward(t(4, 6), t(4, 8), t(6, 8), act="swish")),
    (ValueError, lambda: dense.matmul_backward(t(4, 6), t(4, 8), t(6, 8))),  # not on the GPU
    (TypeError, lambda: dense.matmul_backward(t(4, 6, dtype=F32), t(4, 8), t(6, 8))),
    (TypeError, lambda: moe.route(t(4, 8, dtype=torch.float64), 2)),
    (ValueError, lambda: moe.route(t(4, 8, 1), 2)),
    (ValueError, lambda: moe.route(t(4, 0), 1)),
    (ValueError, lambda: moe.route(t(4, 8), 0)),
    (ValueError, lambda: moe.route(t(4, 8), 9)),
    (ValueError, lambda: moe.route(t(4, 8), 2, score="tanh")),
    (ValueError, lambda: moe.route(t(4, 8), 2)),  # not on the GPU
    (TypeError, lambda: moe.route_backward(t(4, 2, dtype=F32), t(4, 8), t(4, 2, dtype=I64), t(4, 2, dtype=F32))),
    (TypeError, lambda: moe.route_backward(t(4, 2), t(4, 8), t(4, 2, dtype=I32), t(4, 2, dtype=F32))),
    (ValueError, lambda: moe.route_backward(t(4, 3, dtype=F32), t(4, 8), t(4, 2, dtype=I32), t(4, 2, dtype=F32))),
    (ValueError, lambda: moe.route_backward(t(4, 2, dtype=F32), t(5, 8), t(4, 2, dtype=I32), t(4, 2, dtype=F32))),
    (ValueError, lambda: moe.route_backward(t(4, 2, dtype=F32), t(4, 8), t(4, 2, dtype=I32), t(4, 2, dtype=F32), score="max")),
    (TypeError, lambda: layer(dt=F32)),
    (TypeError, lambda: layer(ids_dt=F32)),
    (TypeError, lambda: layer(wt=F16)),
    (TypeError, lambda: layer(wout_dt=BF16)),
    (ValueError, lambda: layer(ids=(5, 2))),
    (ValueError, lambda: layer(ids=(4, 0), weights=(4, 0))),
    (ValueError, lambda: layer(weights=(4, 3))),
    (ValueError, lambda: layer(w_out=(3, 9, 6))),
    (ValueError, lambda: layer(w_out=(0, 8, 6), w_in=(0, 12, 8))),
    (ValueError, lambda: layer(gated=False)),
    (ValueError, lambda: layer(act="glu")),
    (ValueError, lambda: layer()),  # not on the GPU
])
def test_python_refuses(error, call):
    with pytest.raises(error):
        call()


@pytest.mark.parametrize("which", range(5))
def test_the_layer_of_few_tokens_refuses_what_wants_a_gradient(which):
    args = [t(4, 8), t(4, 2, dtype=I32), t(4, 2, dtype=F32), t(3, 12, 8), t(3, 8, 6)]
    if which == 1:
        return
    args[which].requires_grad_(True)
    with pytest.raises(ValueError, match="no gradient"):
        moe.layer(*args)
    with torch.no_grad(), pytest.raises(ValueError, match="on the GPU"):  # none is recorded: on to the next check
        moe.layer(*args)


# each call with its floating tensors, any one of which may carry the tangent
CALLS = [
    ([(4, 8, F16), (6, 8, F16)], lambda x, w: dense.matmul(x, w)),
    ([(4, 6, F16), (4, 8, F16), (6, 8, F16)], lambda dy, x, w: dense.matmul_backward(dy, x, w)),
    ([(4, 8, F32)], lambda l: moe.route(l, 2)),
    ([(4, 2, F32), (4, 8, F32), (4, 2, F32)], lambda d, l, w: moe.route_backward(d, l, t(4, 2, dtype=I32), w)),
    ([(4, 8, F16), (4, 2, F32)], lambda x, w: moe.layer(x, t(4, 2, dtype=I32), w, t(3, 12, 8), t(3, 8, 6))),
]


@pytest.mark.parametrize("shapes,call,which", [(s, c, i) for s, c in CALLS for i in range(len(s))])
def test_tangents_are_refused(shapes, call, which):
    args = [t(*s[:-1], dtype=s[-1]) for s in shapes]
    with fwd.dual_level():
        args[which] = fwd.make_dual(args[which], torch.ones_like(args[which]))
        with torch.no_grad(), pytest.raises(NotImplementedError, match="tangent"):
            call(*args)


@pytest.mark.parametrize("call", [
    lambda: pg.pgemm_dense_run(None, 0, 8, 0, 8, None, None, 0, 0, None, 1, 8, 8, 0, 0, 0, 0),
    lambda: pg.pgemm_dense_backward(None, 0, 8, 0, 8, 0, 8, None, 0, 0, 0, 1, 8, 8, 0, 0, 0, 0),
    lambda: pg.pgemm_moe_route(None, 0, 8, 0, 1, 8, 2, 0, 1, 0, 0),
    lambda: pg.pgemm_moe_route_backward(None, 0, 0, 8, 0, 0, 0, 1, 8, 2, 0, 1, 0),
    lambda: pg.pgemm_moe_layer(None, 0, 8, 0, 0, 0, 0, 0, 0, 1, 2, 3, 8, 6, 0, 0, 0),
])
def test_null_handles_are_refused(call):
    with pytest.raises(pg.PgemmError) as e:
        call()
    assert e.value.status == pg.PGEMM_ERR_INVALID_ARG


def test_workspaces():
    size = pg.pgemm_dense_workspace
    assert size(0, 64, 64, 0) == 0 and size(4, 64, 64, 1) == 0 and size(8192, 8192, 4096, 1) == 0
    assert size(8192, 8192, 4096, 1, wide=False) >= 2 * (8192 * 4096 + 8192 * 4096)  # both operands are moved
    assert size(512, 4096, 8192, 1) >= 4 * 2 * 512 * 4096  # two pieces at least
    back = pg.pgemm_dense_backward_workspace
    assert back(0, 64, 64, 0, 0) >= 0 and back(4096, 1024, 1024, 1, pg.PGEMM_ACT_GELU, 0, 1) >= 2 * 4096 * 1024
    assert back(4096, 1024, 1024, 1, 0, 0, pg.PGEMM_DENSE_DB) < back(4096, 1024, 1024, 1, pg.PGEMM_ACT_SILU, 1, 7)
    few = pg.pgemm_moe_layer_workspace
    assert few(0, 2, 4, 64, 64) == 0 and few(4, 2, 4, 64, 64) > 4 * 2 * 64 * 2
    assert few(64, 2, 4, 64, 64) == few(4096, 2, 4, 64, 64)  # passes of 64 tokens share it
    bad, no = pg.PGEMM_ERR_INVALID_ARG, pg.PGEMM_ERR_UNSUPPORTED
    for call, status in ((lambda: size(-1, 8, 8, 0), bad), (lambda: size(1, 8, 8, 2), bad), (lambda: size(1, 8, 8, 0, 2), bad),
                         (lambda: size(1, 8, 2 ** 22, 0), no), (lambda: size(2 ** 29, 2 ** 20, 8, 0), no),
                         (lambda: back(1, 8, 8, 0, 9), bad), (lambda: back(1, 8, 8, 0, 0, 0, 8), bad),
                         (lambda: few(1, 0, 4, 8, 8), bad), (lambda: few(1, 1, 0, 8, 8), bad), (lambda: few(4097, 1, 4, 8, 8), no),
                         (lambda: few(1, 33, 40, 8, 8), no), (lambda: few(1, 1, 1025, 8, 8), no), (lambda: few(1, 1, 4, 8, 2 ** 20), no)):
        with pytest.raises(pg.PgemmError) as e:
            call()
        assert e.value.status == status


def test_queries_refuse():
    for call in (lambda: pg.pgemm_dense_query(0, 8, 8, 0), lambda: pg.pgemm_dense_query(8, 8, 8, 3),
                 lambda: pg.pgemm_dense_weight_grad_query(8, 0, 8), lambda: pg.pgemm_dense_gradients_query(0, 8, 8, 0),
                 lambda: pg.pgemm_dense_gradients_query(8, 8, 8, 2)):
        with pytest.raises(pg.PgemmError) as e:
            call()
        assert e.value.status == pg.PGEMM_ERR_INVALID_ARG
    with pytest.raises(pg.PgemmError) as e:
        pg.pgemm_dense_query(8, 8, 2 ** 22, 0)
    assert e.value.status == pg.PGEMM_ERR_UNSUPPORTED
