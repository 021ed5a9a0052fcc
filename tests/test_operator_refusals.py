"""CPU: what the routed operators and the 4-bit product refuse, in Python and at the C boundary, before any device work."""
import pytest
import torch

import persistent_tile_scheduling_macro_amd as pg
from persistent_tile_scheduling_macro_amd import moe, w4

F16, BF16, I32 = torch.float16, torch.bfloat16, torch.int32


def t(*shape, dtype=F16):
    return torch.zeros(shape, dtype=dtype)


def plan(n=8, E=3, k=2, dtype=I32):
    return moe.RoutePlan(t(E + 1, dtype=dtype), t(n, dtype=dtype), t(n, dtype=dtype), k)


@pytest.mark.parametrize("error,call", [
    (TypeError, lambda: moe.dispatch(t(4, 8, dtype=torch.float32), t(4, 2, dtype=I32), 3)),
    (ValueError, lambda: moe.dispatch(t(4, 8, 1), t(4, 2, dtype=I32), 3)),
    (TypeError, lambda: moe.dispatch(t(4, 8), t(4, 2), 3)),
    (ValueError, lambda: moe.dispatch(t(4, 8), t(5, 2, dtype=I32), 3)),
    (ValueError, lambda: moe.dispatch(t(4, 8), t(4, 0, dtype=I32), 3)),
    (ValueError, lambda: moe.dispatch(t(4, 8), t(4, dtype=I32), 3)),
    (ValueError, lambda: moe.dispatch(t(4, 8), t(4, 2, dtype=I32), 0)),
    (ValueError, lambda: moe.dispatch(t(4, 8), t(4, 2, dtype=I32), 3)),  # not on the GPU
    (ValueError, lambda: moe.dispatch_backward(t(7, 8), plan())),
    (ValueError, lambda: moe.dispatch_backward(t(8, 8), plan(dtype=torch.int64))),
    (ValueError, lambda: moe.dispatch_backward(t(8, 8), plan(k=3))),
    (ValueError, lambda: moe.dispatch_backward(t(8, 8), plan(k=0))),
    (TypeError, lambda: moe.combine(t(8, 8), t(4, 2), plan())),
    (ValueError, lambda: moe.combine(t(8, 8), t(2, 4, dtype=torch.float32), plan())),
    (ValueError, lambda: moe.combine(t(9, 8), t(4, 2, dtype=torch.float32), plan())),
    (ValueError, lambda: moe.combine_backward(t(3, 8), t(8, 8), t(4, 2, dtype=torch.float32), plan())),
    (TypeError, lambda: moe.combine_backward(t(4, 8, dtype=BF16), t(8, 8), t(4, 2, dtype=torch.float32), plan())),
    (ValueError, lambda: moe.grouped_matmul(t(4, 8), t(2, 6, 8), t(3, dtype=I32), layout="mn")),
    (ValueError, lambda: moe.grouped_matmul(t(4, 8), t(2, 6, 8), t(3, dtype=I32), layout="kn")),
    (ValueError, lambda: moe.grouped_matmul(t(4, 8), t(6, 8), t(3, dtype=I32))),
    (TypeError, lambda: moe.grouped_matmul(t(4, 8), t(2, 6, 8, dtype=BF16), t(3, dtype=I32))),
    (ValueError, lambda: moe.grouped_matmul(t(4, 8), t(2, 6, 8), t(2, dtype=I32))),
    (ValueError, lambda: moe.grouped_matmul(t(4, 8), t(2, 6, 8), t(3, dtype=torch.int64))),
    (ValueError, lambda: moe.grouped_matmul(t(4, 8), t(2, 6, 8), t(3, dtype=I32))),  # not on the GPU
    (ValueError, lambda: moe.grouped_matmul_backward(t(4, 8), t(4, 8), t(2, 6, 8), t(3, dtype=I32))),
    (ValueError, lambda: w4.matmul(t(2, 64), t(8, 32, dtype=torch.uint8), t(8, 2), group=48)),
    (ValueError, lambda: w4.matmul(t(2, 64), t(8, 32, dtype=torch.uint8), t(8, 2), group=32, fmt="int8")),
    (TypeError, lambda: w4.matmul(t(2, 64), t(8, 32, dtype=I32), t(8, 2), group=32)),
    (TypeError, lambda: w4.matmul(t(2, 64), t(8, 32, dtype=torch.uint8), t(8, 2, dtype=BF16), group=32)),
    (ValueError, lambda: w4.matmul(t(2, 64), t(8, 31, dtype=torch.uint8), t(8, 2), group=32)),
    (ValueError, lambda: w4.matmul(t(2, 64), t(8, 32, dtype=torch.uint8), t(8, 1), group=32)),
    (ValueError, lambda: w4.matmul(t(2, 64), t(8, 32, dtype=torch.uint8), t(8, 2), t(8, 2, dtype=torch.uint8), group=32, fmt="e2m1")),
    (TypeError, lambda: w4.matmul(t(2, 64), t(8, 32, dtype=torch.uint8), t(8, 2), t(8, 2), group=32)),
    (ValueError, lambda: w4.matmul(t(2, 64), t(8, 32, dtype=torch.uint8), t(8, 2), t(8, 1, dtype=torch.uint8), group=32)),
    (ValueError, lambda: w4.matmul(t(2, 64), t(3, 8, 32, dtype=torch.uint8), t(3, 8, 2), group=32, offsets=t(3, dtype=I32))),
    (ValueError, lambda: w4.matmul(t(2, 64), t(3, 8, 32, dtype=torch.uint8), t(3, 8, 2), group=32)),
    (ValueError, lambda: w4.matmul(t(2, 64).requires_grad_(True), t(8, 32, dtype=torch.uint8), t(8, 2), group=32)),
    (ValueError, lambda: w4.matmul(t(2, 64), t(8, 32, dtype=torch.uint8), t(8, 2), group=32)),  # not on the GPU
])
def test_python_refuses(error, call):
    with pytest.raises(error):
        call()


@pytest.mark.parametrize("call", [
    lambda: pg.pgemm_moe_dispatch(None, 0, 8, 0, 0, 1, 1, 1, 8, 0, 0, 0, 0, 0),
    lambda: pg.pgemm_moe_dispatch_backward(None, 0, 8, 0, 1, 1, 8, 0, 0),
    lambda: pg.pgemm_moe_combine(None, 0, 8, 0, 0, 1, 1, 8, 0, 0),
    lambda: pg.pgemm_moe_combine_backward(None, 0, 8, 0, 8, 0, 0, 0, 1, 1, 1, 8, 0, 0, 0),
    lambda: pg.pgemm_grouped_run(None, 0, 8, 0, 0, 0, 1, 1, 8, 8, 0, 0),
    lambda: pg.pgemm_grouped_weight_grad(None, 0, 8, 0, 8, 0, 0, 1, 1, 8, 8, 0, 0, 0),
    lambda: pg.pgemm_w4_run(None, 0, 64, 0, 0, 0, 0, 0, 1, 8, 64, 1, 32, 0, 0),
])
def test_null_handles_are_refused(call):
    with pytest.raises(pg.PgemmError) as e:
        call()
    assert e.value.status == pg.PGEMM_ERR_INVALID_ARG


def test_dispatch_workspace():
    assert pg.pgemm_moe_dispatch_workspace(0, 1, 1) == 0 and pg.pgemm_moe_dispatch_workspace(16, 8, 64) == 0
    big = pg.pgemm_moe_dispatch_workspace(8192, 8, 64)
    assert big > 0 and big % 4 == 0
    for args, status in (((-1, 1, 1), pg.PGEMM_ERR_INVALID_ARG), ((1, 0, 1), pg.PGEMM_ERR_INVALID_ARG),
                         ((1, 1, 0), pg.PGEMM_ERR_INVALID_ARG), ((1, 1, 1025), pg.PGEMM_ERR_UNSUPPORTED),
                         ((2 ** 30, 2, 4), pg.PGEMM_ERR_UNSUPPORTED), ((2 ** 40, 1, 4), pg.PGEMM_ERR_UNSUPPORTED)):
        with pytest.raises(pg.PgemmError) as e:
            pg.pgemm_moe_dispatch_workspace(*args)
        assert e.value.status == status


def test_weight_gradient_workspace():
    size = pg.pgemm_grouped_weight_grad_workspace
    assert size(0, 4, 64, 64) == 0 and size(100, 4, 64, 64) == 0 and size(32768, 32, 4096, 2048) == 0
    assert size(32768, 1, 64, 61) % (64 * 64 * 4) == 0 and size(32768, 1, 64, 61) > 0
    for args, status in (((-1, 1, 8, 8), pg.PGEMM_ERR_INVALID_ARG), ((1, 0, 8, 8), pg.PGEMM_ERR_INVALID_ARG),
                         ((1, 1025, 8, 8), pg.PGEMM_ERR_UNSUPPORTED), ((2 ** 31, 1, 8, 8), pg.PGEMM_ERR_UNSUPPORTED)):
        with pytest.raises(pg.PgemmError) as e:
            size(*args)
        assert e.value.status == status
