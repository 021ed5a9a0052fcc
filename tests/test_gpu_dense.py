"""GPU: the linear layer with its epilogue and its gradients, against plain forms in 64 bits."""
import pytest
import torch

import dense_cases as cases
import dense_refs as refs

pytestmark = pytest.mark.gpu

DT = {"f16": torch.float16, "bf16": torch.bfloat16}


@pytest.fixture(scope="module")
def dense():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from persistent_tile_scheduling_macro_amd import dense
    return dense


def inputs(M, N, K, gated, layout, dtype, bias=True, residual=True, seed=1):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, scale=1.0):
        return (torch.randn(shape, generator=g, device="cuda") * scale).to(DT[dtype])

    C = N * (1 + gated)
    fan = max(K, 1) ** -0.5
    w = normal(C, K, scale=fan) if layout == "nk" else normal(K, C, scale=fan)
    return (normal(M, K), w, normal(C, scale=0.5) if bias else None, normal(M, N) if residual else None, normal(M, N))


def check(dense, M, N, K, act, gated, layout, dtype, bias, residual, train=True):
    print(M, N, K, act, gated, layout, dtype, bias, residual, flush=True)
    x, w, b, r, dy = inputs(M, N, K, gated, layout, dtype, bias, residual)
    how = {"act": act, "gated": gated, "layout": layout}
    y, z = dense.matmul(x, w, b, r, preactivation=True, **how)
    assert (z is None) == (act == "none" and not gated)
    refs.check_forward(y, z, x, w, b, r, act, gated, layout)
    assert torch.equal(y, dense.matmul(x, w, b, r, **how))
    if not train:
        return
    dx, dw, db = dense.matmul_backward(dy, x, w, z, need_dbias=True, **how)
    refs.check_backward(dx, dw, db, dy, x, w, z, act, gated, layout)
    for need in ((True, False, False), (False, True, False), (False, False, True)):
        got = dense.matmul_backward(dy, x, w, z, need_dx=need[0], need_dw=need[1], need_dbias=need[2], **how)
        for g, want, n in zip(got, (dx, dw, db), need):
            assert (g is None) == (not n) and (g is None or torch.equal(g, want))


# few rows, tiles of 64 and 128 rows, whole and in pieces, 256 x 256 tiles; even and odd sizes
SIZES = [(1, 256, 512), (1, 40, 33), (5, 72, 131), (8, 512, 1024), (9, 129, 64), (16, 1000, 264), (17, 77, 1001), (32, 264, 4096),
         (33, 136, 200), (64, 512, 2048), (50, 65, 77), (65, 128, 128), (128, 1024, 4096), (200, 1032, 520), (257, 999, 333),
         (512, 520, 1288), (700, 131, 2049), (1500, 2056, 72), (1025, 3000, 1000), (2048, 2048, 256), (4099, 2057, 1021)]


@pytest.mark.parametrize("M,N,K", SIZES)
@pytest.mark.parametrize("layout", ["nk", "kn"])
@pytest.mark.parametrize("act,gated,dtype,bias,residual", [("none", False, "bf16", False, True), ("gelu", False, "f16", True, True),
                                                           ("silu", True, "bf16", False, False),
                                                           ("gelu_tanh", True, "f16", True, True)])
def test_sizes(dense, M, N, K, layout, act, gated, dtype, bias, residual):
    check(dense, M, N, K, act, gated, layout, dtype, bias, residual)


@pytest.mark.parametrize("act", refs.ACTS)
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("M,N,K", [(6, 48, 96), (130, 260, 136)])
def test_activations(dense, act, gated, dtype, M, N, K):
    check(dense, M, N, K, act, gated, "nk", dtype, True, False)


@pytest.mark.parametrize("M", [3, 70])
@pytest.mark.parametrize("act", refs.ACTS)
def test_activations_over_their_range(dense, act, M):
    """An identity as the matrix: every 16-bit value of some range goes through the activation and its slope."""
    for dtype in (torch.float16, torch.bfloat16):
        v = torch.cat([torch.linspace(-30, 30, 64 * M // 2), torch.logspace(-6, 4, 64 * M // 4), -torch.logspace(-6, 4, 64 * M // 4)])
        x = torch.zeros((M, 64), device="cuda")
        x.view(-1)[:v.numel()] = v.cuda()
        x, w = x.to(dtype), torch.eye(64, device="cuda").to(dtype)
        y, z = dense.matmul(x, w, act=act, preactivation=True)
        refs.check_forward(y, z, x, w, None, None, act, False, "nk")
        dy = torch.ones_like(y)
        dx, dw, db = dense.matmul_backward(dy, x, w, z, act=act, need_dbias=True)
        refs.check_backward(dx, dw, db, dy, x, w, z, act, False, "nk")


@pytest.mark.parametrize("M,N,K", [(0, 16, 8), (4, 0, 8), (4, 16, 0), (40, 16, 0), (40, 0, 8), (0, 0, 0), (300, 24, 0)])
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("layout", ["nk", "kn"])
def test_empty_sizes(dense, M, N, K, gated, layout):
    check(dense, M, N, K, "silu", gated, layout, "bf16", True, True)


@pytest.mark.parametrize("M,N,K", [(7, 64, 128), (100, 72, 136), (600, 520, 264)])
@pytest.mark.parametrize("layout", ["nk", "kn"])
def test_views(dense, M, N, K, layout):
    """Rows inside wider ones, at odd addresses, repeated, and a matrix whose rows are not contiguous."""
    x, w, b, r, dy = inputs(M, N, K, False, layout, "bf16")

    def inside(t, left, right):
        wide = torch.full((t.shape[0], t.shape[1] + left + right), float("nan"), dtype=t.dtype, device="cuda")
        wide[:, left:left + t.shape[1]] = t
        return wide[:, left:left + t.shape[1]]

    want, zw = dense.matmul(x, w, b, r, act="gelu", layout=layout, preactivation=True)
    back = dense.matmul_backward(dy, x, w, zw, act="gelu", layout=layout, need_dbias=True)
    for left, right in ((8, 8), (3, 2), (0, 5)):
        args = [inside(t, left, right) for t in (x, w)] + [b, inside(r, left, right)]
        y, z = dense.matmul(*args, act="gelu", layout=layout, preactivation=True)
        assert torch.equal(y, want) and torch.equal(z, zw)
        got = dense.matmul_backward(inside(dy, left, right), *args[:2], z, act="gelu", layout=layout, need_dbias=True)
        for a, c in zip(got, back):
            assert torch.equal(a, c)
    turned = w.t().contiguous().t()
    assert torch.equal(dense.matmul(x, turned, b, r, act="gelu", layout=layout), want)
    one = x[:1].expand(M, K)
    refs.check_forward(dense.matmul(one, w, b, r[:1].expand(M, N), act="gelu", layout=layout), None, one, w, b, r[:1].expand(M, N),
                       "gelu", False, layout)
    g1 = dense.matmul_backward(dy[:1].expand(M, N), one, w, zw, act="gelu", layout=layout, need_dbias=True)
    refs.check_backward(*g1, dy[:1].expand(M, N), one, w, zw, "gelu", False, layout)


@pytest.mark.parametrize("M,N,K", [(5, 37, 96), (65, 96, 75), (300, 200, 190)])
def test_what_lies_around_stays_out(dense, M, N, K):
    """NaN and infinities around the operands reach no output."""
    for dtype in (torch.float16, torch.bfloat16):
        x, w, b, r, dy = inputs(M, N, K, True, "kn", "f16" if dtype == torch.float16 else "bf16")
        want, zw = dense.matmul(x, w, b, r, act="silu", gated=True, layout="kn", preactivation=True)
        back = dense.matmul_backward(dy, x, w, zw, act="silu", gated=True, layout="kn", need_dbias=True)

        def framed(t):
            f = torch.full((t.shape[0] + 2, t.shape[1] + 16), float("inf"), dtype=t.dtype, device="cuda")
            f[1:-1, 8:-8] = t
            return f[1:-1, 8:-8]

        y, z = dense.matmul(framed(x), framed(w), b, framed(r), act="silu", gated=True, layout="kn", preactivation=True)
        assert torch.equal(y, want) and torch.equal(z, zw)
        for a, c in zip(dense.matmul_backward(framed(dy), framed(x), framed(w), z, act="silu", gated=True, layout="kn",
                                              need_dbias=True), back):
            assert torch.equal(a, c)


@pytest.mark.parametrize("M", [4, 200])
@pytest.mark.parametrize("gated", [False, True])
def test_autograd(dense, M, gated):
    N, K = 72, 136
    x, w, b, r, dy = inputs(M, N, K, gated, "nk", "bf16")
    leaves = [t.requires_grad_(True) for t in (x, w, b, r)]
    y = dense.matmul(*leaves, act="silu", gated=gated)
    y.backward(dy)
    with torch.no_grad():
        y2, z = dense.matmul(*leaves, act="silu", gated=gated, preactivation=True)
        want = dense.matmul_backward(dy, x, w, z, act="silu", gated=gated, need_dbias=True)
    assert torch.equal(y, y2)
    for t, g in zip(leaves, (*want, dy)):
        assert torch.equal(t.grad, g)
    only = dense.matmul(x.detach(), w.detach(), b, None, act="silu", gated=gated)
    assert torch.autograd.grad(only, b, dy)[0].equal(want[2])


def test_gradients_against_differences(dense):
    """The directional derivative of a sum of outputs, from fp64 differences of the plain form at the 16-bit inputs."""
    x, w, b, r, dy = inputs(40, 48, 64, True, "nk", "f16", seed=3)
    y, z = dense.matmul(x, w, b, r, act="gelu", gated=True, preactivation=True)
    grads = dense.matmul_backward(dy, x, w, z, act="gelu", gated=True, need_dbias=True)

    def loss(x, w, b):
        z = x @ w.t() + b
        return ((refs.act("gelu", z[:, :48])[0] * z[:, 48:]) * dy.double()).sum()

    at = [t.double() for t in (x, w, b)]
    for i, g in enumerate(grads):
        d = torch.randn(at[i].shape, generator=torch.Generator(device="cuda").manual_seed(i), device="cuda", dtype=torch.float64)
        h = 1e-5
        plus, minus = list(at), list(at)
        plus[i], minus[i] = at[i] + h * d, at[i] - h * d
        numeric = (loss(*plus) - loss(*minus)) / (2 * h)
        # g is off by the roundings of z, dz and itself, three half steps of each element's terms at most
        slack = 6 * 2.0 ** -11 * (g.double().abs() * d.abs()).sum() + 6 * 2.0 ** -11 * g.double().norm() * d.norm()
        assert abs((g.double() * d).sum() - numeric) <= slack


@pytest.mark.parametrize("M,N,K", [(3, 128, 256), (90, 200, 333), (300, 512, 1024)])
def test_graph_capture(dense, M, N, K):
    """Forward and backward captured together, replayed on other inputs between eager calls."""
    x, w, b, r, dy = inputs(M, N, K, True, "nk", "bf16")

    def step():
        y, z = dense.matmul(x, w, b, r, act="silu", gated=True, preactivation=True)
        return y, z, *dense.matmul_backward(dy, x, w, z, act="silu", gated=True, need_dbias=True)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for seed in (5, 6, 7):
        for t, new in zip((x, w, b, r, dy), inputs(M, N, K, True, "nk", "bf16", seed=seed)):
            t.copy_(new)
        graph.replay()
        torch.cuda.synchronize()
        for a, c in zip(out, step()):
            assert torch.equal(a, c)


def test_another_stream(dense):
    x, w, b, r, dy = inputs(300, 256, 512, False, "nk", "f16")
    want = dense.matmul(x, w, b, r, act="gelu")
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = [dense.matmul(x, w, b, r, act="gelu") for _ in range(3)]
    side.synchronize()
    assert all(torch.equal(g, want) for g in got)


@pytest.mark.parametrize("M,N,K,layout,gated,plan", cases.PRODUCTS)
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_every_body(dense, M, N, K, layout, gated, plan, dtype):
    act = "silu" if gated else ("gelu" if M % 2 else "gelu_tanh")
    check(dense, M, N, K, act, gated, layout, dtype, True, True, train=False)


@pytest.mark.parametrize("M,N,K,plan", cases.GRADIENTS)
@pytest.mark.parametrize("layout,dtype", [("nk", "f16"), ("kn", "bf16")])
def test_every_body_of_the_weight_gradient(dense, M, N, K, plan, layout, dtype):
    print(M, N, K, layout, dtype, flush=True)
    if layout == "kn":  # dw is [K, N] there: the same tiles
        N, K = K, N
    x, w, _, _, dy = inputs(M, N, K, False, layout, dtype)
    _, dw, _ = dense.matmul_backward(dy, x, w, layout=layout, need_dx=False)
    refs.check_backward(None, dw, None, dy, x, w, None, "none", False, layout)


@pytest.mark.parametrize("M,N,K,layout,plan", cases.BOTH)
@pytest.mark.parametrize("act,dtype", [("none", "f16"), ("silu", "bf16")])
def test_both_gradients(dense, M, N, K, layout, plan, act, dtype):
    print(M, N, K, layout, act, dtype, flush=True)
    x, w, b, _, dy = inputs(M, N, K, False, layout, dtype)
    _, z = dense.matmul(x, w, b, act=act, layout=layout, preactivation=True)
    dx, dw, db = dense.matmul_backward(dy, x, w, z, act=act, layout=layout, need_dbias=True)
    refs.check_backward(dx, dw, db, dy, x, w, z, act, False, layout)


@pytest.mark.parametrize("N,K", [(1, 1), (1, 64), (2, 9), (3, 200), (4, 40), (7, 7), (9, 3)])
@pytest.mark.parametrize("M", [1, 20, 200])
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("layout", ["nk", "kn"])
def test_narrow_matrices(dense, M, N, K, gated, layout):
    check(dense, M, N, K, "gelu", gated, layout, "f16", True, True)


@pytest.mark.parametrize("M", [3, 300])
def test_infinities_and_nan_stay_in_their_rows(dense, M):
    x, w, b, r, dy = inputs(M, 72, 64, True, "nk", "bf16")
    want, zw = dense.matmul(x, w, b, r, act="silu", gated=True, preactivation=True)
    dxw, _, _ = dense.matmul_backward(dy, x, w, zw, act="silu", gated=True, need_dw=False)
    x2, dy2 = x.clone(), dy.clone()
    x2[1, 5], dy2[2, 3] = float("inf"), float("nan")
    y, z = dense.matmul(x2, w, b, r, act="silu", gated=True, preactivation=True)
    dx, _, _ = dense.matmul_backward(dy2, x, w, zw, act="silu", gated=True, need_dw=False)
    other = [i for i in range(M) if i != 1]
    assert not bool(y[1].isfinite().all()) and torch.equal(y[other], want[other]) and torch.equal(z[other], zw[other])
    other = [i for i in range(M) if i != 2]
    assert bool(dx[2].isnan().all()) and torch.equal(dx[other], dxw[other])


@pytest.mark.parametrize("act", ["none", "relu", "gelu", "gelu_tanh", "silu"])
@pytest.mark.parametrize("M", [2, 200])
def test_infinite_sums(dense, act, M):
    x = torch.ones(M, 64, device="cuda", dtype=torch.bfloat16)
    x[1, 3] = float("inf")
    y = dense.matmul(x, torch.ones(80, 64, device="cuda", dtype=torch.bfloat16), act=act)
    assert bool((y[1] == float("inf")).all()) and bool(y[0].isfinite().all())


def test_large_gradients_are_read_past_the_cache(dense):
    """The activation's gradient of more bytes than the memory-side cache holds."""
    check(dense, 8200, 7176, 24, "gelu", False, "nk", "bf16", True, False)


def test_a_layer_feeds_a_router_and_the_experts(dense):
    """Training through the linear layer, the router and the routed operators: each node's gradient is its operator's own."""
    from persistent_tile_scheduling_macro_amd import moe
    T, H, I, E, k = 96, 128, 72, 6, 2
    g = torch.Generator(device="cuda").manual_seed(4)

    def normal(*shape, scale=1.0):
        return (torch.randn(shape, generator=g, device="cuda") * scale).bfloat16().requires_grad_(True)

    x, w_x, router = normal(T, H), normal(2 * H, H, scale=H ** -0.5), normal(E, H, scale=H ** -0.5)
    w_in, w_out = normal(E, I, H, scale=H ** -0.5), normal(E, H, I, scale=I ** -0.5)
    leaves = (x, w_x, router, w_in, w_out)
    dout = torch.randn((T, H), generator=g, device="cuda").bfloat16()

    def step():
        h = dense.matmul(x, w_x, None, x, act="silu", gated=True)
        ids, weights = moe.route(dense.matmul(h, router), k)
        rows, plan = moe.dispatch(h, ids, E)
        out = moe.combine(moe.grouped_matmul(moe.grouped_matmul(rows, w_in, plan.offsets), w_out, plan.offsets), weights, plan)
        return (out.detach(),) + torch.autograd.grad(out, leaves, dout)

    def by_hand():
        with torch.no_grad():
            h, z = dense.matmul(x, w_x, None, x, act="silu", gated=True, preactivation=True)
            logits = dense.matmul(h, router)
            ids, weights = moe.route(logits, k)
            rows, plan = moe.dispatch(h, ids, E)
            up = moe.grouped_matmul(rows, w_in, plan.offsets)
            down = moe.grouped_matmul(up, w_out, plan.offsets)
            out = moe.combine(down, weights, plan)
            ddown, dweights = moe.combine_backward(dout, down, weights, plan)
            dup, dw_out = moe.grouped_matmul_backward(ddown, up, w_out, plan.offsets)
            drows, dw_in = moe.grouped_matmul_backward(dup, rows, w_in, plan.offsets)
            dlogits = moe.route_backward(dweights, logits, ids, weights)
            dh1, drouter, _ = dense.matmul_backward(dlogits, h, router)
            dh2 = moe.dispatch_backward(drows, plan)
            dh = dh1 + dh2
            dx, dw_x, _ = dense.matmul_backward(dh, x, w_x, z, act="silu", gated=True)
            return out, dx + dh, dw_x, drouter, dw_in, dw_out

    want = by_hand()
    for a, b in zip(step(), want):
        assert torch.equal(a, b) or (a.double() - b.double()).norm() <= 2.0 ** -7 * b.double().norm()  # sums of two in either order
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        captured = step()
    for _ in range(3):
        with torch.no_grad():
            x.copy_(torch.randn((T, H), generator=g, device="cuda").bfloat16())
        eager = step()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(captured, eager):
            assert torch.equal(a, b)


@pytest.mark.parametrize("gated", [False, True])
def test_offsets_past_32_bits(dense, gated):
    """More than 2^31 elements of y, z and dz: their last rows and columns."""
    M, N, K = 66001, 33000 // (1 + gated), 24
    x, w, _, _, dy = inputs(M, N, K, gated, "nk", "bf16", False, False)
    y, z = dense.matmul(x, w, act="silu", gated=gated, preactivation=True)
    assert z.numel() > 2 ** 31
    refs.check_forward(y[-70:], z[-70:], x[-70:], w, None, None, "silu", gated, "nk")
    dx, dw, _ = dense.matmul_backward(dy, x, w, z, act="silu", gated=gated)
    refs.check_backward(dx[-70:], None, None, dy[-70:], x[-70:], w, z[-70:], "silu", gated, "nk")
    if not gated:
        refs.check_backward(None, dw[-8:], None, dy[:, -8:], x, w[-8:], z[:, -8:], "silu", False, "nk")
