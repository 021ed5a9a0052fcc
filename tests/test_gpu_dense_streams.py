"""GPU: the linear layer, the router and the routed layer on two streams at once, and two captured graphs of one pool."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def calls():
    """Each operator where it takes a workspace or joins pieces, as a function of a seed's inputs."""
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from persistent_tile_scheduling_macro_amd import dense, moe
    g = torch.Generator(device="cuda").manual_seed(11)

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda").bfloat16() * 0.25

    w, w_odd, w_in, w_out = normal(520, 4096), normal(77, 301), normal(5, 2 * 40, 2056), normal(5, 2056, 40)
    b = normal(520)

    def product(x):
        return dense.matmul(x, w, b, act="gelu", preactivation=True)

    def gradient(x):
        y, z = dense.matmul(x, w, b, act="gelu", preactivation=True)
        return dense.matmul_backward(y, x, w, z, act="gelu", need_dbias=True)

    def odd(x):
        part = x[:, :301]
        return dense.matmul_backward(dense.matmul(part, w_odd), part, w_odd)[:2]

    def route(x):
        ids, weights = moe.route(x[:, :200], 6, score="sigmoid")
        return ids, weights, moe.route_backward(weights, x[:, :200], ids, weights, score="sigmoid")

    def layer(x):
        ids, weights = moe.route(x[:, :5], 2)
        return (moe.layer(x[:, :2056], ids, weights, w_in, w_out),)

    return {"product": product, "gradient": gradient, "odd": odd, "route": route, "layer": layer}


def rows(seed, T=100):
    return torch.randn((T, 4096), generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda").bfloat16()


@pytest.mark.parametrize("name", ["product", "gradient", "odd", "route", "layer"])
def test_two_streams_at_once(calls, name):
    call = calls[name]
    x = [rows(1), rows(2)]
    want = [call(v) for v in x]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[], []]
    for _ in range(10):
        for i in (0, 1):
            with torch.cuda.stream(streams[i]):
                got[i].append(call(x[i]))
    torch.cuda.synchronize()
    for i in (0, 1):
        for outputs in got[i]:
            assert all(torch.equal(a, b) for a, b in zip(outputs, want[i]))


@pytest.mark.parametrize("name", ["product", "gradient", "odd", "route", "layer"])
def test_two_graphs_of_one_pool(calls, name):
    call = calls[name]
    x = [rows(3), rows(4)]
    for v in x:
        call(v)
    torch.cuda.synchronize()
    graphs, outputs = [torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()], []
    pool = torch.cuda.graph_pool_handle()
    for graph, v in zip(graphs, x):
        with torch.cuda.graph(graph, pool=pool):
            outputs.append(call(v))
    for turn in range(3):
        for v in x:
            v.copy_(rows(10 + turn))
        want = [call(v) for v in x]
        for i in ((0, 1), (1, 0), (0, 1))[turn]:
            graphs[i].replay()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(outputs[i], want[i]))


@pytest.mark.parametrize("name", ["product", "gradient", "odd", "route", "layer"])
def test_no_rows_change_when_others_do(calls, name):
    """Each row's results depend on that row alone, to the bit, where the count of rows stays."""
    if name in ("gradient", "odd"):  # dw and dbias sum over rows: their dx alone
        call = lambda v: calls[name](v)[:1]
    else:
        call = calls[name]
    a, b = rows(5, 40), rows(6, 40)
    b[7] = a[7]
    for x, y in zip(call(a), call(b)):
        assert torch.equal(x[7], y[7])
