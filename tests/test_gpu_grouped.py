"""GPU: products of rows sorted by expert against plain forms in 64 bits.

Sizes cover every path of the rule that picks a kernel: operands at 16-byte
addresses and at odd ones, both layouts, few and many rows per expert, empty
experts and rows of none. Small whole numbers make every sum exact, so there
the gradients have to equal differences exactly.
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


def normal(*shape, dtype, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda").to(dtype)


def operands(counts, K, N, layout, dtype, before=0, after=0, seed=1):
    off = ref.offsets_of(counts, before)
    R = before + sum(counts) + after
    x = normal(R, K, dtype=dtype, seed=seed)
    w = normal(len(counts), *((K, N) if layout == "kn" else (N, K)), dtype=dtype, seed=seed + 1)
    dy = normal(R, N, dtype=dtype, seed=seed + 2)
    return x, w, dy, off


def check_all(moe, x, w, dy, off, layout, what):
    print(what, flush=True)
    K, most = x.shape[1], int((off[1:] - off[:-1]).max())
    y = moe.grouped_matmul(x, w, off, layout=layout)
    dx, dw = moe.grouped_matmul_backward(dy, x, w, off, layout=layout)
    torch.cuda.synchronize()
    ref.assert_within(y, *ref.grouped(x, w, off, layout), K, f"y {what}")
    ref.assert_within(dx, *ref.grouped(dy, w, off, "nk" if layout == "kn" else "kn"), dy.shape[1], f"dx {what}")
    a, b = (x, dy) if layout == "kn" else (dy, x)
    ref.assert_within(dw, *ref.grouped_dw(a, b, off), most, f"dw {what}")
    none = torch.ones(x.shape[0], dtype=torch.bool, device="cuda")
    none[int(off[0]):int(off[-1])] = False
    assert not bool(y[none].any()) and not bool(dx[none].any())


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("layout", ["kn", "nk"])
@pytest.mark.parametrize("counts,K,N", [
    ([1], 1, 1), ([1], 64, 64), ([0, 1, 0], 8, 8), ([3, 0, 2], 7, 5), ([17, 16, 15], 128, 96), ([5, 9, 1, 0, 33], 200, 72),
    ([130, 0, 127, 128], 136, 264), ([64, 65, 63], 65, 129), ([300, 1, 40], 520, 136), ([257, 255, 256, 511], 256, 512),
    ([700, 300], 1000, 264), ([513, 90], 1001, 257), ([2, 1, 3, 2], 2047, 130), ([9, 7], 2048, 8),
    ([90, 0, 3, 1], 136, 200), ([0, 0, 70, 0], 257, 131), ([20, 32, 33], 7, 5), ([32], 128, 128), ([31, 33], 264, 6)])
def test_products_and_gradients(moe, counts, K, N, layout, dtype):
    check_all(moe, *operands(counts, K, N, layout, DT[dtype]), layout, f"{counts} {K}x{N} {layout} {dtype}")


@pytest.mark.parametrize("layout", ["kn", "nk"])
@pytest.mark.parametrize("counts,K,N", [([1500], 40, 24), ([4100], 64, 64), ([3000, 10, 0], 33, 47), ([5000, 3], 136, 7),
                                        ([1, 2600], 200, 72), ([0, 900, 2000], 5, 264), ([2049], 131, 135)])
def test_weight_gradients_over_many_rows(moe, counts, K, N, layout):
    """Few output tiles: the rows are cut into pieces, of every length with uneven experts."""
    for dtype in DT.values():
        check_all(moe, *operands(counts, K, N, layout, dtype, after=2), layout, f"{counts} {K}x{N} {layout} {dtype}")


@pytest.mark.parametrize("layout", ["kn", "nk"])
@pytest.mark.parametrize("counts,K,N", [([5, 3], 64, 72), ([200, 150], 136, 264), ([600, 700], 264, 512), ([40, 9], 33, 17)])
def test_rows_of_no_expert_give_zeros(moe, counts, K, N, layout):
    x, w, dy, off = operands(counts, K, N, layout, torch.bfloat16, before=3, after=131)
    for t in (x, dy):  # what they hold never matters
        t[:3] = float("nan")
        t[3 + sum(counts):] = float("inf")
    check_all(moe, x, w, dy, off, layout, f"gaps {counts} {K}x{N} {layout}")


@pytest.mark.parametrize("R", [0, 1, 40, 300])
def test_no_rows_for_any_expert(moe, R):
    x, w = normal(R, 64, dtype=torch.float16, seed=1), normal(4, 64, 72, dtype=torch.float16, seed=2)
    dy, off = normal(R, 72, dtype=torch.float16, seed=3), torch.zeros(5, dtype=torch.int32, device="cuda")
    y = moe.grouped_matmul(x, w, off, layout="kn")
    dx, dw = moe.grouped_matmul_backward(dy, x, w, off, layout="kn")
    assert y.shape == (R, 72) and dx.shape == (R, 64) and dw.shape == (4, 64, 72)
    assert not bool(y.any()) and not bool(dx.any()) and not bool(dw.any())


@pytest.mark.parametrize("layout", ["kn", "nk"])
def test_empty_sides(moe, layout):
    off = ref.offsets_of([2, 3])
    for K, N in ((0, 16), (16, 0), (0, 0)):
        x, w, dy, off = operands([2, 3], K, N, layout, torch.bfloat16)
        y = moe.grouped_matmul(x, w, off, layout=layout)
        dx, dw = moe.grouped_matmul_backward(dy, x, w, off, layout=layout)
        assert y.shape == (5, N) and dx.shape == (5, K) and dw.shape == w.shape
        assert not bool(y.any()) and not bool(dx.any())


@pytest.mark.parametrize("layout", ["kn", "nk"])
def test_nan_and_infinity_stay_in_their_rows(moe, layout):
    """A row's sum runs over all its elements and no other row's, whatever the tiles round up to."""
    for counts, K, N in (([7, 9], 72, 40), ([130, 140], 72, 136), ([300, 290], 200, 264)):
        x, w, dy, off = operands(counts, K, N, layout, torch.bfloat16)
        want = moe.grouped_matmul(x, w, off, layout=layout)
        x[counts[0]:] = float("nan")  # all of the second expert's
        got = moe.grouped_matmul(x, w, off, layout=layout)
        assert torch.equal(got[:counts[0]], want[:counts[0]]) and bool(got[counts[0]:].isnan().all())
        dw = moe.grouped_matmul_backward(dy, x, w, off, layout=layout, need_dx=False)[1]
        assert not bool(dw[0].isnan().any()) and bool(dw[1].isnan().all())


@pytest.mark.parametrize("layout", ["kn", "nk"])
@pytest.mark.parametrize("counts", [[6, 0, 10], [150, 131], [300, 280]])
def test_strides(moe, layout, counts):
    """Rows that are slices of wider ones, at even and odd places, and one row repeated."""
    K, N = 72, 136
    for lead, width in ((8, 96), (3, 96), (1, 77)):
        x, w, dy, off = operands(counts, K, N, layout, torch.float16)
        big = normal(x.shape[0], width, dtype=torch.float16, seed=9)
        big[:, lead:lead + K] = x
        wide = normal(x.shape[0], N + 40, dtype=torch.float16, seed=10)
        wide[:, lead:lead + N] = dy
        check_all(moe, big[:, lead:lead + K], w, wide[:, lead:lead + N], off, layout, f"slice {lead} of {width}")
    check_all(moe, x[:1].expand(x.shape[0], K), w, dy[:1].expand(x.shape[0], N), off, layout, "one row")
    flat = torch.empty(w.numel() + 1, dtype=w.dtype, device="cuda")  # a matrix at an odd address
    flat[1:] = w.reshape(-1)
    check_all(moe, x, flat[1:].view(w.shape), dy, off, layout, "odd address")
    check_all(moe, x.t().contiguous().t(), w.transpose(1, 2).contiguous().transpose(1, 2), dy, off, layout, "transposed")


@pytest.mark.parametrize("layout", ["kn", "nk"])
@pytest.mark.parametrize("counts", [[3, 4, 0, 1], [140, 0, 150], [300, 270]])
def test_whole_numbers_are_exact_and_gradients_equal_differences(moe, layout, counts):
    K, N = 40, 24
    g = torch.Generator(device="cuda").manual_seed(3)

    def whole(*shape):
        return torch.randint(-1, 2, shape, generator=g, device="cuda").to(torch.bfloat16)

    R, E = sum(counts), len(counts)
    x, dy, off = whole(R, K), whole(R, N), ref.offsets_of(counts)
    w = whole(E, *((K, N) if layout == "kn" else (N, K)))
    y = moe.grouped_matmul(x, w, off, layout=layout)
    assert torch.equal(y.double(), ref.grouped(x, w, off, layout)[0])
    dx, dw = moe.grouped_matmul_backward(dy, x, w, off, layout=layout)

    def loss(x, w):
        return (moe.grouped_matmul(x, w, off, layout=layout).double() * dy.double()).sum()

    for leaf, grad, args in ((x, dx, lambda t: (t, w)), (w, dw, lambda t: (x, t))):
        for i in torch.randint(0, leaf.numel(), (6,), generator=g, device="cuda").tolist():
            up, down = leaf.clone(), leaf.clone()
            up.view(-1)[i] += 1
            down.view(-1)[i] -= 1
            d = (loss(*args(up)) - loss(*args(down))) / 2
            assert grad.reshape(-1)[i].double() == d or abs(float(d)) > 256, i


def test_autograd(moe):
    x, w, dy, off = operands([70, 0, 60], 96, 80, "nk", torch.bfloat16)
    dx, dw = moe.grouped_matmul_backward(dy, x, w, off, layout="nk")
    for gx, gw in ((True, True), (True, False), (False, True)):
        xl, wl = x.clone().requires_grad_(gx), w.clone().requires_grad_(gw)
        moe.grouped_matmul(xl, wl, off, layout="nk").backward(dy)
        assert (xl.grad is None) != gx and (wl.grad is None) != gw
        assert not gx or torch.equal(xl.grad, dx)
        assert not gw or torch.equal(wl.grad, dw)
    xl = x.clone().requires_grad_(True)
    moe.grouped_matmul(xl, w, off, layout="nk").sum().backward()  # a gradient of stride 0
    want = moe.grouped_matmul_backward(torch.ones_like(dy), x, w, off, layout="nk", need_dw=False)[0]
    assert torch.equal(xl.grad, want)


@pytest.mark.parametrize("counts,K,N", [([4, 5, 6], 256, 128), ([200, 190, 30], 264, 136), ([800, 300], 512, 520), ([33, 2], 77, 31),
                                        ([2000, 700], 72, 40)])
def test_graph_replays_with_other_bounds(moe, counts, K, N):
    """Captured once, replayed with other offsets and rows, eager work between: each replay equals the eager call."""
    x, w, dy, off = operands(counts, K, N, "nk", torch.bfloat16)

    def step():
        return (moe.grouped_matmul(x, w, off, layout="nk"),) + moe.grouped_matmul_backward(dy, x, w, off, layout="nk")

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    R = sum(counts)
    for i in range(4):
        cuts = sorted(torch.randint(0, R + 1, (len(counts) - 1,), generator=torch.Generator().manual_seed(i)).tolist())
        off.copy_(torch.tensor([0] + cuts + [R], dtype=torch.int32))
        x.copy_(normal(R, K, dtype=x.dtype, seed=20 + i))
        want = step()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(out, want):
            assert torch.equal(a, b), i


def test_another_stream(moe):
    x, w, dy, off = operands([90, 300], 256, 264, "kn", torch.float16)
    want = moe.grouped_matmul(x, w, off, layout="kn")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        x2 = x * 1
        got = moe.grouped_matmul(x2, w, off, layout="kn")
    s.synchronize()
    assert torch.equal(got, want)


def test_rows_past_32_bit_offsets(moe):
    """x, its gradient and one expert's place in w lie more than 2^32 bytes into their tensors."""
    R, K, N = 1050000, 2056, 8
    x = torch.zeros((R, K), dtype=torch.bfloat16, device="cuda")
    x[-40:] = normal(40, K, dtype=x.dtype, seed=1)
    w = normal(2, N, K, dtype=x.dtype, seed=2)
    off = torch.tensor([0, R - 30, R], dtype=torch.int32, device="cuda")
    y = moe.grouped_matmul(x, w, off, layout="nk")
    tail = ref.grouped(x[-40:], w, torch.tensor([0, 10, 40]), "nk")
    ref.assert_within(y[-40:], *tail, K, "y")
    assert not bool(y[:-40].any())
    dy = torch.zeros((R, N), dtype=x.dtype, device="cuda")
    dy[-40:] = normal(40, N, dtype=x.dtype, seed=3)
    dx, dw = moe.grouped_matmul_backward(dy, x, w, off, layout="nk")
    ref.assert_within(dx[-40:], *ref.grouped(dy[-40:], w, torch.tensor([0, 10, 40]), "kn"), N, "dx")
    ref.assert_within(dw, *ref.grouped_dw(dy[-40:], x[-40:], torch.tensor([0, 10, 40])), 30, "dw")


@pytest.mark.parametrize("rows", [1, 200])
def test_matrices_past_32_bit_offsets(moe, rows):
    E, K, N = 70, 8192, 4096
    w = torch.zeros((E, K, N), dtype=torch.float16, device="cuda")
    w[-1] = normal(K, N, dtype=w.dtype, seed=1) / 64
    x = normal(rows, K, dtype=w.dtype, seed=2)
    off = torch.full((E + 1,), 0, dtype=torch.int32, device="cuda")
    off[-1] = rows
    y = moe.grouped_matmul(x, w, off, layout="kn")
    ref.assert_within(y, *ref.grouped(x, w[-1:], torch.tensor([0, rows]), "kn"), K, "y")


def test_many_experts(moe):
    g = torch.Generator().manual_seed(5)
    counts = torch.randint(0, 4, (1000,), generator=g).tolist()
    check_all(moe, *operands(counts, 24, 40, "kn", torch.bfloat16), "kn", "1000 experts")
    counts = [0] * 1024
    counts[1023], counts[511] = 150, 2
    check_all(moe, *operands(counts, 64, 72, "nk", torch.bfloat16), "nk", "1024 experts, two in use")


def test_bounds_that_do_not_fit_stay_inside(moe):
    """Offsets that lie outside the rows or run backwards read and write nothing past a tensor's end."""
    x, w, dy, _ = operands([300, 200, 12], 64, 72, "nk", torch.bfloat16)
    for bad in ([0, 100, 9000, 9000], [-5, 100, 200, 300], [300, 200, 100, 0], [2147483647, 0, -2147483648, 512]):
        off = torch.tensor(bad, dtype=torch.int32, device="cuda")
        y = moe.grouped_matmul(x, w, off, layout="nk")
        dx, dw = moe.grouped_matmul_backward(dy, x, w, off, layout="nk")
        torch.cuda.synchronize()
        assert y.shape == (512, 72) and dx.shape == (512, 64) and dw.shape == w.shape
