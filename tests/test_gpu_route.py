"""GPU: the router and its gradient, against plain forms in 64 bits.

Bounds: an fp32 exponential of a difference of logits is off by the difference's rounding, |l - max| * 2^-24 relative, and
a few steps of 2^-23; a sum of E positive terms by E steps at most. A gradient multiplies a few such factors.
"""
import pytest
import torch

from dense_refs import outside
import operator_refs as ref

pytestmark = pytest.mark.gpu

INF = float("inf")
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


@pytest.fixture(scope="module")
def moe():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from persistent_tile_scheduling_macro_amd import moe
    return moe


def logits_of(T, E, dtype, masked=0.0, empty=0.0, seed=1, scale=1.5):
    g = torch.Generator(device="cuda").manual_seed(seed)
    l = torch.randn((T, E), generator=g, device="cuda") * scale
    closed = (torch.rand((T, E), generator=g, device="cuda") < masked) | (torch.rand((T, 1), generator=g, device="cuda") < empty)
    return l.masked_fill(closed, -INF).to(TYPES[dtype])


def plain(logits, k, score, normalize, dweights=None):
    """(ids, weights, their relative error, gradient, its error) in 64 bits; NaN logits count as -inf."""
    l = logits.double().masked_fill(logits.isnan(), -INF)
    E = l.shape[1]
    top, ids = torch.sort(l, dim=1, descending=True, stable=True)
    top, ids = top[:, :k], ids[:, :k]
    live = top > -INF
    most = torch.where(live[:, :1], top[:, :1], 0.0)
    if score == "softmax":
        s = torch.exp(l - most)
        s = s / s.sum(1, keepdim=True).clamp(min=1e-300)
        eps = (E + 16 + (l - most).abs().clamp(max=200)) * 2.0 ** -23
    else:
        s = torch.sigmoid(l)
        eps = (E + 16 + (l - most).abs().clamp(max=200) * normalize) * 2.0 ** -23
    hot = torch.zeros_like(l).scatter_(1, ids, live.double())
    share = s * hot
    if normalize:  # in logarithms, where the scores themselves underflow
        log = torch.where(hot > 0, l if score == "softmax" else torch.nn.functional.logsigmoid(l), -INF)
        share = torch.softmax(log, 1).nan_to_num(nan=0.0)
    w = torch.where(live, share.gather(1, ids), 0.0)
    chosen = torch.where(live, ids, -1).int()
    we = eps.gather(1, ids)
    if dweights is None:
        return chosen, w, we
    d = torch.zeros_like(l).scatter_(1, ids, torch.where(live, dweights.double(), 0.0))
    mean, size = (share * d).sum(1, keepdim=True), (share * d).abs().sum(1, keepdim=True)
    if score == "softmax" and not normalize:
        grad, err = s * (d - mean), s * (d.abs() + size)
    elif score == "softmax":
        grad, err = share * (d - mean), share * (d.abs() + size)
    else:
        f = share * torch.sigmoid(-l)
        grad, err = f * (d - mean * (1.0 if normalize else 0.0)), f * (d.abs() + size)
    return chosen, w, we, grad, 4 * eps * err


def check(moe, logits, k, score, normalize):
    how = {"score": score, "normalize": normalize}
    ids, weights = moe.route(logits, k, **how)
    g = torch.Generator(device="cuda").manual_seed(9)
    dweights = torch.randn(weights.shape, generator=g, device="cuda")
    dweights[ids < 0] = float("nan")
    chosen, w, we, grad, err = plain(logits, k, score, normalize, dweights)
    assert ids.dtype == torch.int32 and torch.equal(ids, chosen)
    assert weights.dtype == torch.float32
    outside(weights, w, we * w + 2.0 ** -126, "weights")
    got = moe.route_backward(dweights, logits, ids, weights, **how)
    assert got.dtype == logits.dtype
    outside(got, grad, err + ref.HALF[got.dtype] * (grad.abs() + err) + max(ref.TINY[got.dtype], 2.0 ** -126), "dlogits")


SIZES = [(1, 1, 1), (1, 2, 2), (3, 7, 3), (16, 64, 8), (33, 8, 8), (100, 13, 3), (65, 16, 16), (257, 33, 4), (40, 32, 32),
         (129, 65, 6), (500, 128, 8), (64, 200, 64), (300, 256, 8), (90, 257, 9), (70, 512, 8), (31, 1000, 64), (17, 1024, 40),
         (4099, 13, 3), (9000, 64, 6)]


@pytest.mark.parametrize("T,E,k", SIZES)
@pytest.mark.parametrize("dtype,masked,empty", [("f32", 0.0, 0.0), ("bf16", 0.3, 0.1), ("f16", 0.9, 0.0)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("normalize", [False, True])
def test_sizes(moe, T, E, k, dtype, masked, empty, score, normalize):
    print(T, E, k, dtype, score, normalize, flush=True)
    check(moe, logits_of(T, E, dtype, masked, empty), k, score, normalize)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("normalize", [False, True])
def test_values(moe, score, normalize):
    """Equal logits, zeros of both signs, the type's extremes, infinities, NaN."""
    rows = [[0.0] * 6, [-0.0, 0.0, -0.0, 0.0, 0.0, -0.0], [1.0, 2.0, 2.0, 1.0, 2.0, 0.5], [-INF] * 6, [-INF, -INF, 3.0, -INF, 3.0, -INF],
            [float("nan"), 1.0, float("nan"), -INF, 0.0, -1.0], [-65504.0, 65504.0, 0.0, 1.0, -1.0, 65504.0],
            [float("nan")] * 6, [-65504.0] * 6, [80.0, -80.0, 79.0, -81.0, 80.0, 0.0], [6e-8, -6e-8, 0.0, 1e-7, -INF, 1e-7]]
    for dtype in TYPES.values():
        check(moe, torch.tensor(rows, device="cuda").to(dtype), 4, score, normalize)
    lowest = torch.full((3, 5), torch.finfo(torch.float32).min, device="cuda")
    lowest[1, 2] = 0.0
    check(moe, lowest, 3, score, normalize)


def test_infinite_logits_give_nan_weights_and_their_ids(moe):
    ids, w = moe.route(torch.tensor([[0.0, INF, 1.0]], device="cuda"), 2)
    assert ids.tolist() == [[1, 2]] and bool(w.isnan().all())


@pytest.mark.parametrize("E", [5, 64, 300])
def test_views(moe, E):
    l = logits_of(50, E, "bf16", 0.2, 0.1)
    for left, right in ((1, 3), (0, 8)):
        wide = torch.full((50, E + left + right), 100.0, dtype=l.dtype, device="cuda")
        wide[:, left:left + E] = l
        v = wide[:, left:left + E]
        for a, b in zip(moe.route(v, 4), moe.route(l, 4)):
            assert torch.equal(a, b)
        check(moe, v, 4, "softmax", False)
    for a, b in zip(moe.route(l.t().contiguous().t(), 4), moe.route(l, 4)):
        assert torch.equal(a, b)
    check(moe, l[:1].expand(50, E), 4, "sigmoid", True)


def test_no_tokens(moe):
    ids, w = moe.route(torch.empty((0, 8), device="cuda"), 3)
    assert ids.shape == w.shape == (0, 3)
    assert moe.route_backward(w, torch.empty((0, 8), device="cuda"), ids, w).shape == (0, 8)


def test_autograd_and_differences(moe):
    l = logits_of(40, 24, "f32", 0.2, 0.1).requires_grad_(True)
    for score in ("softmax", "sigmoid"):
        for normalize in (False, True):
            ids, w = moe.route(l, 5, score=score, normalize=normalize)
            assert not ids.requires_grad and w.requires_grad
            d = torch.randn(w.shape, generator=torch.Generator(device="cuda").manual_seed(2), device="cuda")
            (grad,) = torch.autograd.grad(w, l, d)
            assert torch.equal(grad, moe.route_backward(d, l.detach(), ids, w.detach(), score=score, normalize=normalize))
            v = torch.randn(l.shape, generator=torch.Generator(device="cuda").manual_seed(3), device="cuda", dtype=torch.float64)
            h, at = 1e-6, l.detach().double()
            live = at > -INF
            step = torch.where(live, h * v, 0.0)  # a step this small changes no choice

            def loss(x):
                s = torch.softmax(x, 1).nan_to_num() if score == "softmax" else torch.sigmoid(x)
                s = torch.where(ids >= 0, s.gather(1, ids.clamp(min=0).long()), 0.0)
                if normalize:
                    s = s / s.sum(1, keepdim=True).clamp(min=1e-300)
                return (s * d.double()).sum()

            numeric = (loss(at + step) - loss(at - step)) / (2 * h)
            terms = (grad.double() * torch.where(live, v, 0.0))
            assert abs(terms.sum() - numeric) <= 1e-4 * terms.abs().sum()


def test_graph_capture(moe):
    l = logits_of(100, 48, "bf16")
    d = torch.randn((100, 6), device="cuda")

    def step():
        ids, w = moe.route(l, 6, normalize=False)
        return ids, w, moe.route_backward(d, l, ids, w, normalize=False)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for seed in (3, 4, 5):
        l.copy_(logits_of(100, 48, "bf16", 0.5, 0.2, seed=seed))
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(out, step()):
            assert torch.equal(a, b)
