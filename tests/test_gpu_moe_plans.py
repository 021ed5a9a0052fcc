"""GPU: gradients under a plan from which slots were taken after the sort (their pos set to a place outside the rows)."""
import pytest
import torch

import operator_refs as ref
from test_gpu_moe import DT, gen, moe, normal, routing  # noqa: F401 (moe is the fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,k,E,H,drop", [(20, 3, 4, 64, 0.0), (1, 1, 1, 1, 0.0), (700, 8, 16, 33, 0.2), (513, 4, 7, 2056, 0.1),
                                          (9000, 2, 5, 40, 0.0), (40, 8, 64, 1021, 0.5), (70000, 4, 16, 24, 0.05)])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("share", [0.3, 1.0])
def test_rows_of_slots_taken_out_get_no_gradient(moe, T, k, E, H, drop, dtype, share):  # noqa: F811
    """out does not depend on such a row of ys, so its gradient is zero, whatever memory held before."""
    print(T, k, E, H, dtype, share, flush=True)
    offsets, order, pos = ref.sort_slots(routing(T, k, E, drop), E)
    out = torch.rand(T * k, generator=gen(3), device="cuda") < share
    n = T * k
    bad = torch.tensor([-1, n, 2 ** 31 - 1, -2 ** 31], dtype=torch.int64, device="cuda")[torch.arange(n, device="cuda") % 4]
    pos = torch.where(out, bad, pos.long()).to(torch.int32)
    plan = moe.RoutePlan(offsets, order, pos, k)
    ys, w, dout = normal(n, H, dtype=DT[dtype], seed=1), torch.rand((T, k), generator=gen(2), device="cuda"), normal(T, H, dtype=DT[dtype], seed=5)
    want = torch.zeros((n, H), dtype=torch.float64, device="cuda")
    at = torch.nonzero((pos >= 0) & (pos < n)).reshape(-1)
    want[pos[at].long()] = dout[at // k].double() * w.reshape(-1)[at].double()[:, None]
    for _ in range(3):  # the allocator hands out a block that held NaN
        del_me = torch.full((n, H), float("nan"), dtype=DT[dtype], device="cuda")
        del del_me
        dys, dw = moe.combine_backward(dout, ys, w, plan)
        ref.assert_within(dys, want, want.abs(), 1, "dys")
    leaf = ys.clone().requires_grad_(True)
    moe.combine(leaf, w, plan).backward(dout)
    assert torch.equal(leaf.grad, dys)


def test_a_plan_needs_its_order(moe):  # noqa: F811
    import persistent_tile_scheduling_macro_amd as pg
    h, b = pg.pgemm_create(0), torch.zeros(1 << 12, dtype=torch.uint8, device="cuda")
    with pytest.raises(pg.PgemmError) as e:
        pg.pgemm_moe_combine_backward_plan(h, b, 8, b, 8, b, b, None, b, 2, 2, 3, 8, pg.PGEMM_F16, b, b)
    assert e.value.status == pg.PGEMM_ERR_INVALID_ARG
    pg.pgemm_moe_combine_backward_plan(h, None, 8, None, 8, None, None, None, None, 0, 2, 3, 8, pg.PGEMM_F16, None, None)
    pg.pgemm_destroy(h)


def test_no_order_on_the_host(moe):  # noqa: F811
    plan = moe.RoutePlan(*ref.sort_slots(routing(4, 2, 3), 3), 2)
    plan.order = plan.order.cpu()
    y = normal(8, 16, dtype=torch.float16, seed=1)
    with pytest.raises(ValueError):
        moe.combine_backward(y[:4], y, torch.rand((4, 2), device="cuda"), plan)
