"""GPU: token rows to their experts and back, against plain forms in 64 bits.

Covers both forms of the sort (one launch, three launches), rows at even and
odd addresses, dropped slots whatever their weights and rows hold, and the
layer made of dispatch, the grouped products and combine with its gradients.
"""
import pytest
import torch

import operator_refs as ref

pytestmark = pytest.mark.gpu

DT = {"f16": torch.float16, "bf16": torch.bfloat16}


@pytest.fixture(scope="module")
def moe():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from persistent_tile_scheduling_macro_amd import moe
    return moe


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def normal(*shape, dtype, seed):
    return torch.randn(shape, generator=gen(seed), device="cuda").to(dtype)


def routing(T, k, E, drop=0.0, seed=1, dtype=torch.int64):
    ids = torch.randint(0, E, (T, k), generator=gen(seed), device="cuda")
    away = torch.rand((T, k), generator=gen(seed + 1), device="cuda") < drop
    return torch.where(away, torch.where(ids % 2 == 0, -1, E), ids).to(dtype)


def check_plan(plan, ids, E):
    for got, want, what in zip((plan.offsets, plan.order, plan.pos), ref.sort_slots(ids, E), ("offsets", "order", "pos")):
        assert got.dtype == torch.int32 and torch.equal(got, want), what


def sorted_rows(x, order, k):
    xs = torch.zeros((order.numel(), x.shape[1]), dtype=x.dtype, device=x.device)
    at = torch.nonzero(order >= 0).reshape(-1)
    xs[at] = x[order[at].long() // k]
    return xs


SIZES = [(1, 1, 1, 1), (1, 8, 8, 64), (3, 2, 4, 7), (17, 3, 13, 72), (64, 8, 64, 1021), (256, 8, 8, 64), (257, 8, 16, 33),
         (300, 11, 40, 136), (2048, 1, 5, 24), (2049, 1, 1024, 24), (700, 9, 1000, 2056), (1500, 4, 3, 1032), (5, 20, 7, 2049),
         (4096, 4, 300, 40), (5461, 3, 1024, 16), (4097, 4, 64, 40), (9000, 8, 200, 24)]


@pytest.mark.parametrize("T,k,E,H", SIZES)
@pytest.mark.parametrize("dtype,ids_dtype,drop", [("f16", torch.int32, 0.0), ("bf16", torch.int64, 0.3), ("bf16", torch.int32, 1.0)])
def test_dispatch_and_its_gradient(moe, T, k, E, H, dtype, ids_dtype, drop):
    print(T, k, E, H, dtype, drop, flush=True)
    x, ids = normal(T, H, dtype=DT[dtype], seed=5), routing(T, k, E, drop, dtype=ids_dtype)
    xs, plan = moe.dispatch(x, ids, E)
    check_plan(plan, ids, E)
    assert torch.equal(xs, sorted_rows(x, plan.order, k))
    dxs = normal(T * k, H, dtype=DT[dtype], seed=6)
    dxs[int(plan.offsets[-1]):] = float("nan")  # rows of no slot
    dx = moe.dispatch_backward(dxs, plan)
    rows = ref.slot_rows(dxs, plan.pos, k)
    ref.assert_within(dx, rows.sum(1), rows.abs().sum(1), k, "dx")


@pytest.mark.parametrize("T,k,E,H", SIZES)
@pytest.mark.parametrize("dtype,drop", [("f16", 0.0), ("bf16", 0.3), ("f16", 1.0)])
def test_combine_and_its_gradients(moe, T, k, E, H, dtype, drop):
    print(T, k, E, H, dtype, drop, flush=True)
    ids = routing(T, k, E, drop)
    plan = moe.RoutePlan(*ref.sort_slots(ids, E), k)
    kept, n = int(plan.offsets[-1]), T * k
    ys, w = normal(n, H, dtype=DT[dtype], seed=7), torch.rand((T, k), generator=gen(8), device="cuda")
    dout = normal(T, H, dtype=DT[dtype], seed=9)
    dropped = plan.pos.view(T, k) < 0
    ys[kept:] = float("inf")
    w[dropped] = float("nan")
    out = moe.combine(ys, w, plan)
    dys, dw = moe.combine_backward(dout, ys, w, plan)
    rows = ref.slot_rows(ys, plan.pos, k)
    wd = torch.where(dropped, 0.0, w.double())[:, :, None]
    ref.assert_within(out, (rows * wd).sum(1), (rows * wd).abs().sum(1), k, "out")
    want = torch.zeros((n, H), dtype=torch.float64, device="cuda")
    at = torch.nonzero(plan.pos >= 0).reshape(-1)
    want[plan.pos[at].long()] = dout[at // k].double() * w.reshape(-1)[at].double()[:, None]
    ref.assert_within(dys, want, want.abs(), 1, "dys")
    assert not bool(dys[kept:].any())
    prod = rows * dout.double()[:, None]
    ref.assert_within(dw, prod.sum(2), prod.abs().sum(2), H, "dw")
    assert not bool(dw[dropped].any())


@pytest.mark.parametrize("T", [4, 400])
def test_ids_far_outside_are_dropped(moe, T):
    k, E, H = 6, 5, 16
    ids = routing(T, k, E)
    far = torch.tensor([2 ** 32 + 1, -2 ** 63, 2 ** 63 - 1, -2 ** 32, E, -1], device="cuda")
    ids[::2] = far
    x = normal(T, H, dtype=torch.float16, seed=1)
    xs, plan = moe.dispatch(x, ids, E)
    check_plan(plan, ids, E)
    assert torch.equal(xs, sorted_rows(x, plan.order, k))


@pytest.mark.parametrize("T", [9, 600])
def test_one_expert_takes_all(moe, T):
    ids = torch.full((T, 4), 6, dtype=torch.int32, device="cuda")
    x = normal(T, 40, dtype=torch.bfloat16, seed=1)
    xs, plan = moe.dispatch(x, ids, 8)
    check_plan(plan, ids, 8)
    assert torch.equal(xs, x.repeat_interleave(4, 0))


def test_empty_batches(moe):
    for T, k, H in ((0, 2, 16), (3, 2, 0), (0, 1, 0)):
        x = torch.zeros((T, H), dtype=torch.float16, device="cuda")
        ids = torch.zeros((T, k), dtype=torch.int64, device="cuda")
        w = torch.rand((T, k), device="cuda")
        xs, plan = moe.dispatch(x, ids, 4)
        check_plan(plan, ids, 4)
        out = moe.combine(xs, w, plan)
        dys, dw = moe.combine_backward(out, xs, w, plan)
        assert xs.shape == (T * k, H) and out.shape == (T, H) and dys.shape == xs.shape and dw.shape == w.shape
        assert moe.dispatch_backward(xs, plan).shape == (T, H) and not bool(dw.any())


@pytest.mark.parametrize("T,H", [(40, 72), (900, 1024), (500, 1032)])
def test_strides(moe, T, H):
    k, E = 4, 6
    ids, w = routing(T, k, E, 0.2), torch.rand((T, k), generator=gen(1), device="cuda")
    wide = normal(T * k, H + 11, dtype=torch.bfloat16, seed=2)
    for lead in (0, 1, 8):
        xv, yv, dv = wide[:T, lead:lead + H], wide[:, lead:lead + H], wide[1:1 + T, lead:lead + H]
        xs, plan = moe.dispatch(xv, ids.t().contiguous().t(), E)
        assert torch.equal(xs, sorted_rows(xv.contiguous(), plan.order, k))
        assert torch.equal(moe.combine(yv, w, plan), moe.combine(yv.contiguous(), w, plan))
        for a, b in zip(moe.combine_backward(dv, yv, w, plan), moe.combine_backward(dv.contiguous(), yv.contiguous(), w, plan)):
            assert torch.equal(a, b)
        assert torch.equal(moe.dispatch_backward(yv, plan), moe.dispatch_backward(yv.contiguous(), plan))
    one = wide[:1, :H]
    xs, plan = moe.dispatch(one.expand(T, H), ids, E)
    assert torch.equal(xs, sorted_rows(one.repeat(T, 1), plan.order, k))
    got, want = moe.combine_backward(one.expand(T, H), yv, w, plan), moe.combine_backward(one.repeat(T, 1), yv, w, plan)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    xt = wide[:T, :H].t().contiguous().t()  # columns that are contiguous instead: copied first
    assert torch.equal(moe.dispatch(xt, ids, E)[0], sorted_rows(wide[:T, :H], plan.order, k))


def test_positions_that_do_not_fit_count_as_dropped(moe):
    T, k, H = 20, 3, 64
    plan = moe.RoutePlan(*ref.sort_slots(routing(T, k, 4), 4), k)
    ys, w, dout = normal(T * k, H, dtype=torch.float16, seed=1), torch.rand((T, k), device="cuda"), normal(T, H, dtype=torch.float16, seed=2)
    bad = plan.pos.clone()
    bad[::5] = torch.tensor([T * k, -7, 2147483647, -2147483648], dtype=torch.int32, device="cuda").repeat(3)
    gone = plan.pos.clone()
    gone[::5] = -1
    a, b = moe.RoutePlan(plan.offsets, plan.order, bad, k), moe.RoutePlan(plan.offsets, plan.order, gone, k)
    assert torch.equal(moe.combine(ys, w, a), moe.combine(ys, w, b))
    assert torch.equal(moe.combine_backward(dout, ys, w, a)[1], moe.combine_backward(dout, ys, w, b)[1])


@pytest.mark.parametrize("T,k,E", [(30, 2, 4), (1100, 2, 6)])
def test_gradients_equal_differences(moe, T, k, E):
    """Whole numbers and weights in quarters: every value is exact, so differences are too."""
    H, g = 40, gen(4)

    def whole(*shape):
        return torch.randint(-3, 4, shape, generator=g, device="cuda").to(torch.bfloat16)

    x, ids = whole(T, H), routing(T, k, E, 0.2)
    xs, plan = moe.dispatch(x, ids, E)
    w = torch.randint(-4, 5, (T, k), generator=g, device="cuda").float() / 4
    dxs, ys, dout = whole(T * k, H), whole(T * k, H), whole(T, H)
    dx, (dys, dw) = moe.dispatch_backward(dxs, plan), moe.combine_backward(dout, ys, w, plan)

    def there(x):
        return (moe.dispatch(x, ids, E)[0].double() * dxs.double()).sum()

    def back(ys, w):
        return (moe.combine(ys, w, plan).double() * dout.double()).sum()

    for leaf, grad, f in ((x, dx, there), (ys, dys, lambda t: back(t, w)), (w, dw, lambda t: back(ys, t))):
        for i in torch.randint(0, leaf.numel(), (8,), generator=g, device="cuda").tolist():
            up, down = leaf.clone(), leaf.clone()
            up.view(-1)[i] += 1
            down.view(-1)[i] -= 1
            assert grad.reshape(-1)[i].double() == (f(up) - f(down)) / 2, i


def layer(moe, x, ids, w1, w2, weights, E):
    xs, plan = moe.dispatch(x, ids, E)
    hidden = torch.relu(moe.grouped_matmul(xs, w1, plan.offsets, layout="kn"))
    return moe.combine(moe.grouped_matmul(hidden, w2, plan.offsets, layout="nk"), weights, plan)


@pytest.mark.parametrize("T,H,F", [(60, 64, 96), (1500, 72, 136)])
def test_a_layer_and_its_gradients(moe, T, H, F):
    """Whole numbers again: the layer's result and every gradient equal those of the plain form in 64 bits."""
    E, k, g = 5, 2, gen(11)

    def sparse(*shape, p=0.06):
        sign = torch.randint(0, 2, shape, generator=g, device="cuda") * 2 - 1
        return (sign * (torch.rand(shape, generator=g, device="cuda") < p)).to(torch.bfloat16)

    ids = routing(T, k, E, 0.1)
    leaves = [sparse(T, H, p=0.2), sparse(E, H, F), sparse(E, H, F), torch.randint(-1, 2, (T, k), generator=g, device="cuda").float()]
    dout = sparse(T, H, p=0.1)
    mine = [t.clone().requires_grad_(True) for t in leaves]
    out = layer(moe, mine[0], ids, mine[1], mine[2], mine[3], E)
    out.backward(dout)
    plain = [t.double().requires_grad_(True) for t in leaves]
    want = torch.zeros((T, H), dtype=torch.float64, device="cuda")
    for e in range(E):
        share = (plain[3] * (ids == e)).sum(1, keepdim=True)
        want = want + share * (torch.relu(plain[0] @ plain[1][e]) @ plain[2][e].t())
    want.backward(dout.double())
    assert float(want.detach().abs().max()) < 256 and torch.equal(out.detach().double(), want.detach())
    for a, b in zip(mine, plain):
        assert float(b.grad.abs().max()) > 0
        fits = b.grad.abs() <= 256  # whole numbers up to 256 have eight bits
        assert torch.equal(a.grad.double()[fits], b.grad[fits])


def test_autograd_leaves_out_what_needs_no_gradient(moe):
    x, ids = normal(30, 64, dtype=torch.float16, seed=1).requires_grad_(True), routing(30, 2, 4)
    xs, plan = moe.dispatch(x, ids, 4)
    assert xs.requires_grad and not plan.offsets.requires_grad
    xs.sum().backward()
    assert torch.equal(x.grad, torch.full_like(x, 2.0))
    with torch.no_grad():
        assert not moe.dispatch(x, ids, 4)[0].requires_grad
    w = torch.rand((30, 2), device="cuda", requires_grad=True)
    moe.combine(xs.detach(), w, plan).sum().backward()
    assert w.grad is not None


@pytest.mark.parametrize("T", [12, 800])
def test_graph_replays_with_other_routes(moe, T):
    """One capture of the steps and their gradients; every replay, eager work between, equals the eager calls."""
    E, k, H, F = 6, 3, 72, 40
    x, ids, weights = normal(T, H, dtype=torch.bfloat16, seed=1), routing(T, k, E, 0.1), torch.rand((T, k), generator=gen(2), device="cuda")
    w, dout = normal(E, F, H, dtype=torch.bfloat16, seed=3), normal(T, F, dtype=torch.bfloat16, seed=4)

    def step():
        xs, plan = moe.dispatch(x, ids, E)
        ys = moe.grouped_matmul(xs, w, plan.offsets)
        out = moe.combine(ys, weights, plan)
        dys, dw = moe.combine_backward(dout, ys, weights, plan)
        dxs, dm = moe.grouped_matmul_backward(dys, xs, w, plan.offsets)
        return out, dw, dm, moe.dispatch_backward(dxs, plan), plan.offsets, plan.pos

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for i in range(4):
        ids.copy_(routing(T, k, E, 0.2, seed=30 + i))
        x.copy_(normal(T, H, dtype=x.dtype, seed=40 + i))
        want = step()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(out, want):
            assert torch.equal(a, b), i


def test_another_stream(moe):
    x, ids = normal(700, 264, dtype=torch.float16, seed=1), routing(700, 4, 9)
    want, plan = moe.dispatch(x, ids, 9)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got, other = moe.dispatch(x * 1, ids, 9)
    s.synchronize()
    assert torch.equal(got, want) and torch.equal(other.pos, plan.pos)


def test_rows_past_32_bit_offsets(moe):
    T, k, E, H = 66000, 8, 16, 4104  # 4.3 GB of sorted rows
    x = normal(1, H, dtype=torch.bfloat16, seed=1).expand(T, H) * torch.ones((T, 1), dtype=torch.bfloat16, device="cuda")
    x[:, 0] = torch.arange(T, device="cuda") % 251
    ids = routing(T, k, E, 0.01, dtype=torch.int32)
    xs, plan = moe.dispatch(x, ids, E)
    at = torch.nonzero(plan.order >= 0).reshape(-1)
    assert torch.equal(xs[at, 0], x[plan.order[at].long() // k, 0])
    assert torch.equal(xs[at[-1000:]], x[plan.order[at[-1000:]].long() // k]) and not bool(xs[at.numel():].any())
    w = torch.ones((T, k), device="cuda")
    out = moe.combine(xs, w, plan)
    kept = (plan.pos.view(T, k) >= 0).sum(1)
    want = x[-500:].double() * kept[-500:, None]
    ref.assert_within(out[-500:], want, want.abs(), k, "out")
    dys, dw = moe.combine_backward(x, xs, w, plan)
    assert torch.equal(dys, xs)
    dots = (x[-500:].double() ** 2).sum(1, keepdim=True) * (plan.pos.view(T, k)[-500:] >= 0)
    ref.assert_within(dw[-500:], dots, dots, H, "dw")
