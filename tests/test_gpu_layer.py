"""GPU: the routed layer of few tokens, against a plain form in 64 bits and against its parts."""
import pytest
import torch

import dense_refs as refs
import operator_refs as ref

pytestmark = pytest.mark.gpu

DT = {"f16": torch.float16, "bf16": torch.bfloat16}


@pytest.fixture(scope="module")
def moe():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from persistent_tile_scheduling_macro_amd import moe
    return moe


def inputs(T, k, E, H, I, gated, dtype, drop=0.0, distinct=True, ids_type=torch.int32, seed=1):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, scale=1.0):
        return (torch.randn(shape, generator=g, device="cuda") * scale).to(DT[dtype])

    if distinct and k <= E:
        ids = torch.rand((T, E), generator=g, device="cuda").topk(k, dim=1).indices
    else:
        ids = torch.randint(0, E, (T, k), generator=g, device="cuda")
    away = torch.rand((T, k), generator=g, device="cuda") < drop
    ids = torch.where(away, torch.where(ids % 2 == 0, -1, E + 5), ids).to(ids_type)
    weights = torch.rand((T, k), generator=g, device="cuda") + 0.1
    weights[(ids < 0) | (ids >= E)] = float("nan")
    return (normal(T, H), ids, weights, normal(E, I * (1 + gated), H, scale=max(H, 1) ** -0.5), normal(E, H, I, scale=max(I, 1) ** -0.5))


def check(out, x, ids, weights, w_in, w_out, act, gated):
    T, H = x.shape
    I = w_out.shape[2]
    E = w_out.shape[0]
    want = torch.zeros((T, H), dtype=torch.float64, device="cuda")
    err, terms = torch.zeros_like(want), torch.zeros_like(want)
    for e in range(E):
        hit = ids == e
        rows = torch.nonzero(hit.any(1)).reshape(-1)
        if rows.numel() == 0:
            continue
        share = torch.where(hit[rows], weights[rows].double(), 0.0).sum(1, keepdim=True)
        xd, wd = x[rows].double(), w_in[e].double().t().contiguous()
        z, off = xd @ wd, H * 2.0 ** -23 * (xd.abs() @ wd.abs())
        value, _, eps = refs.act(act, z[:, :I])
        e_h = refs.MOST_SLOPE * off[:, :I] + eps * value.abs() + refs.FLUSHED * z[:, :I].abs()
        if gated:
            e_h = e_h * (z[:, I:].abs() + off[:, I:]) + value.abs() * off[:, I:]
            value = value * z[:, I:]
            e_h = e_h + 2.0 ** -24 * value.abs()
        e_h = e_h + ref.HALF[x.dtype] * (value.abs() + e_h) + ref.TINY[x.dtype]  # h in 16 bits
        o = w_out[e].double().t().contiguous()
        want[rows] += share * (value @ o)
        size = share.abs() * ((value.abs() + e_h) @ o.abs())
        err[rows] += share.abs() * (e_h @ o.abs()) + 4 * 2.0 ** -24 * size  # the sum of an expert's weights, its product
        terms[rows] += size
    slots = ids.shape[1]
    err = err + (I + slots + 8) * 2.0 ** -23 * terms
    refs.outside(out, want, err + ref.HALF[out.dtype] * (want.abs() + err) + ref.TINY[out.dtype], "out")


SIZES = [(1, 1, 1, 64, 64), (1, 8, 64, 256, 128), (3, 2, 5, 33, 17), (8, 4, 6, 136, 72), (9, 3, 13, 1021, 517), (11, 3, 13, 1000, 520),
         (16, 8, 16, 512, 256), (17, 2, 4, 200, 333), (24, 8, 300, 64, 96), (32, 4, 8, 1024, 512), (33, 5, 7, 129, 65),
         (40, 2, 2, 512, 264), (64, 8, 64, 320, 192), (64, 32, 40, 72, 40), (64, 1, 1024, 48, 40), (65, 2, 4, 128, 64), (5, 2, 3, 40, 7), (20, 2, 3, 7, 5), (50, 3, 5, 9, 1), (4, 2, 3, 1, 8), (3, 4, 90, 64, 8),
         (6, 2, 4, 4104, 72), (36, 6, 21, 286, 1500), (46, 3, 9, 944, 600), (2, 2, 6, 16, 4000), (64, 4, 4, 100, 1000), (127, 2, 5, 80, 700), (60, 2, 3, 72, 2100), (20, 8, 90, 130, 300), (30, 2, 4, 264, 3500), (30, 4, 100, 4096, 136), (64, 3, 7, 4100, 65),
         (150, 6, 12, 96, 100)]


@pytest.mark.parametrize("T,k,E,H,I", SIZES)
@pytest.mark.parametrize("act,gated,dtype,drop,ids_type", [("silu", True, "bf16", 0.0, torch.int32), ("gelu", False, "f16", 0.3, torch.int64),
                                                           ("gelu_tanh", True, "f16", 0.0, torch.int64)])
def test_sizes(moe, T, k, E, H, I, act, gated, dtype, drop, ids_type):
    print(T, k, E, H, I, act, gated, dtype, flush=True)
    a = inputs(T, k, E, H, I, gated, dtype, drop, ids_type=ids_type)
    out = moe.layer(*a, act=act, gated=gated)
    check(out, *a, act, gated)
    assert torch.equal(out, moe.layer(*a, act=act, gated=gated))


@pytest.mark.parametrize("T", [4, 30, 64])
@pytest.mark.parametrize("act", refs.ACTS)
def test_experts_named_twice(moe, T, act):
    a = inputs(T, 6, 3, 104, 88, False, "bf16", 0.2, distinct=False)
    check(moe.layer(*a, act=act, gated=False), *a, act, False)


@pytest.mark.parametrize("T", [1, 20, 64, 70])
def test_no_slot_left(moe, T):
    a = inputs(T, 2, 4, 64, 48, True, "f16", drop=1.1)
    assert not bool(moe.layer(*a).any())


@pytest.mark.parametrize("T,H,I", [(0, 64, 32), (4, 0, 32), (4, 64, 0)])
def test_empty_sizes(moe, T, H, I):
    a = inputs(T, 2, 4, H, I, True, "bf16")
    out = moe.layer(*a)
    assert out.shape == (T, H) and not bool(out.any())


@pytest.mark.parametrize("T,k,E", [(5, 1, 9), (64, 1, 9), (64, 1, 300), (63, 2, 40), (128, 1, 300), (30, 3, 500)])
def test_one_expert_takes_all(moe, T, k, E):
    """Groups of every size, several of one expert among them; with k > 1 the others go to one each."""
    a = list(inputs(T, k, E, 136, 200, True, "bf16"))
    a[1][:, 0] = 7
    a[1][:, 1:] = a[1][:, 1:].clamp(min=8)
    check(moe.layer(*a), *a, "silu", True)


def test_ids_far_outside_are_dropped(moe):
    a = list(inputs(6, 6, 5, 64, 64, True, "f16", ids_type=torch.int64, distinct=False))
    a[1][::2] = torch.tensor([2 ** 32 + 1, -2 ** 63, 2 ** 63 - 1, -2 ** 32, 5, -1], device="cuda")
    a[2][::2] = float("nan")
    check(moe.layer(*a), *a, "silu", True)


@pytest.mark.parametrize("T", [3, 40])
def test_views_and_rows_of_nobody(moe, T):
    """Rows inside wider ones; NaN in tokens without an expert and in experts without a token."""
    x, ids, weights, w_in, w_out = inputs(T, 2, 8, 72, 40, True, "bf16")
    ids[T // 2] = -1
    x[T // 2] = float("nan")
    weights[T // 2] = float("nan")
    ids[ids == 3] = 4
    w_in[3], w_out[3] = float("nan"), float("inf")
    want = moe.layer(x, ids, weights, w_in, w_out)
    assert not bool(want[T // 2].any()) and bool(want.isfinite().all())
    for left, right in ((8, 8), (3, 2)):
        wide = torch.full((T, 72 + left + right), float("inf"), dtype=x.dtype, device="cuda")
        wide[:, left:left + 72] = x
        assert torch.equal(moe.layer(wide[:, left:left + 72], ids, weights, w_in, w_out), want)
    assert torch.equal(moe.layer(x, ids.t().contiguous().t(), weights.t().contiguous().t(), w_in, w_out), want)


@pytest.mark.parametrize("T", [2, 48])
def test_like_its_parts(moe, T):
    """The router, the layer, and the same layer of dispatch, grouped products and combine, as near as their roundings let them be."""
    from persistent_tile_scheduling_macro_amd import dense
    x, _, _, w_in, w_out = inputs(T, 2, 16, 256, 192, True, "bf16")
    router = torch.randn((16, 256), generator=torch.Generator(device="cuda").manual_seed(5), device="cuda").bfloat16() / 16
    ids, weights = moe.route(dense.matmul(x, router), 4)
    out = moe.layer(x, ids, weights, w_in, w_out)
    check(out, x, ids, weights, w_in, w_out, "silu", True)
    xs, plan = moe.dispatch(x, ids, 16)
    gate, up = moe.grouped_matmul(xs, w_in, plan.offsets).float().chunk(2, 1)
    parts = moe.combine(moe.grouped_matmul((gate * torch.sigmoid(gate) * up).bfloat16(), w_out, plan.offsets), weights, plan)
    # z, h and the experts' outputs are rounded on the way there: three half steps of a bf16 value more
    assert (out.double() - parts.double()).norm() <= 4 * 2.0 ** -8 * out.double().norm()


@pytest.mark.parametrize("T", [3, 64])
def test_graph_capture(moe, T):
    a = inputs(T, 3, 12, 128, 72, True, "bf16", 0.1)
    moe.layer(*a)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = moe.layer(*a)
    for seed in (2, 3, 4):
        for t, new in zip(a, inputs(T, 3, 12, 128, 72, True, "bf16", 0.4, seed=seed)):
            t.copy_(new)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, moe.layer(*a))


def test_offsets_past_32_bits(moe):
    """Matrices of more than 2^31 elements: the last experts."""
    a = list(inputs(3, 2, 130, 4100, 2070, True, "bf16"))
    a[3] = torch.cat([a[3], a[3][-4:]])  # with copies of the last ones
    a[4] = torch.cat([a[4], a[4][-4:]])
    assert a[3].numel() > 2 ** 31
    a[1][:] = torch.tensor([[133, 0], [132, 131], [130, 133]], device="cuda")
    check(moe.layer(*a), *a, "silu", True)


def test_the_most_tokens(moe):
    """4096 tokens go in 64 passes through one workspace."""
    a = list(inputs(4096, 3, 9, 72, 40, True, "f16", drop=0.1))
    check(moe.layer(*a), *a, "silu", True)
