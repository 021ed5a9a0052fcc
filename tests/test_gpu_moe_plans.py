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


GUARD = 4096


class Guarded:
    """Outputs inside buffers of a value that no result here has; untouched() looks at what lies around them."""

    def __init__(self):
        self.flats = []

    def __call__(self, *shape, dtype):
        n = torch.Size(shape).numel()
        flat = torch.full((n + 2 * GUARD,), 777, dtype=dtype, device="cuda")
        self.flats.append((flat, n))
        return flat[GUARD:GUARD + n].view(shape)

    def untouched(self):
        return all(bool((f[:GUARD] == 777).all()) and bool((f[GUARD + n:] == 777).all()) for f, n in self.flats)


@pytest.mark.parametrize("T,k,E,H", [(3, 2, 4, 7), (250, 8, 64, 72), (2049, 1, 1024, 24), (700, 9, 1000, 2056), (1500, 4, 3, 1031),
                                     (33000, 8, 5, 1032)])  # the last one's rows pass the memory-side cache
def test_outputs_end_where_they_end(moe, T, k, E, H):  # noqa: F811
    """Every output of the routing steps, guarded on both sides, with ids, positions and bounds that do not fit."""
    import persistent_tile_scheduling_macro_amd as pg
    print(T, k, E, H, flush=True)
    h, n, f, i32 = pg.pgemm_create(0), T * k, torch.bfloat16, torch.int32
    pg.pgemm_set_stream(h, torch.cuda.current_stream())
    ids = routing(T, k, E, 0.2)
    x, ys, w = normal(T, H, dtype=f, seed=1), normal(n, H, dtype=f, seed=2), torch.rand((T, k), generator=gen(3), device="cuda")
    out = Guarded()
    offsets, order, pos, xs = out(E + 1, dtype=i32), out(n, dtype=i32), out(n, dtype=i32), out(n, H, dtype=f)
    need = pg.pgemm_moe_dispatch_workspace(T, k, E)
    work = out(max(need // 4, 1), dtype=i32)
    pg.pgemm_moe_dispatch(h, x, H, ids, pg.PGEMM_IDS_I64, T, k, E, H, pg.PGEMM_BF16, offsets, order, pos, xs, work, need)
    torch.cuda.synchronize()
    want, plan = moe.dispatch(x, ids, E)
    assert out.untouched() and torch.equal(xs, want) and torch.equal(pos, plan.pos) and torch.equal(offsets, plan.offsets)
    wild = pos.clone()
    wild[::3] = torch.tensor([n, -5, 2 ** 31 - 1, -2 ** 31], dtype=i32, device="cuda")[torch.arange(wild[::3].numel(), device="cuda") % 4]
    far = order.clone()
    far[1::4] = torch.tensor([n, -5, 2 ** 31 - 1, -2 ** 31], dtype=i32, device="cuda")[torch.arange(far[1::4].numel(), device="cuda") % 4]
    for p, o, off in ((pos, order, offsets), (wild, order, offsets), (wild, far, offsets), (pos, order, torch.full_like(offsets, 2 ** 31 - 1)),
                      (pos, order, torch.full_like(offsets, -2 ** 31))):
        out = Guarded()
        dx, back, dys, dw = out(T, H, dtype=f), out(T, H, dtype=f), out(n, H, dtype=f), out(T, k, dtype=torch.float32)
        pg.pgemm_moe_dispatch_backward(h, ys, H, p, T, k, H, pg.PGEMM_BF16, dx)
        pg.pgemm_moe_combine(h, ys, H, w, p, T, k, H, pg.PGEMM_BF16, back)
        pg.pgemm_moe_combine_backward_plan(h, x, H, ys, H, w, off, o, p, T, k, E, H, pg.PGEMM_BF16, dys, dw)
        torch.cuda.synchronize()
        assert out.untouched()
        rows = ref.slot_rows(ys, torch.where((p >= 0) & (p < n), p, -1), k)
        ref.assert_within(dx, rows.sum(1), rows.abs().sum(1), k, "dx")
        wd = w.double()[:, :, None]
        ref.assert_within(back, (rows * wd).sum(1), (rows * wd).abs().sum(1), k, "out")
        prod = rows * x.double()[:, None]
        ref.assert_within(dw, prod.sum(2), prod.abs().sum(2), H, "dw")
        del rows, prod
        assert not bool((dys == 777).any()) or off is not offsets  # every row is written under the sort's bounds
    pg.pgemm_destroy(h)
