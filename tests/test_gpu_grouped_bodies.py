"""GPU: every body of the grouped products, in both layouts and types, against plain forms in 64 bits.

The sizes are those of operator_cases.py, which name the body they take; test_operator_coverage.py holds them to it. Each
goes through uneven and empty experts, rows of none, NaN in one expert, replay with other bounds, rows of wider tensors,
and bounds that do not fit. Whole numbers make sums exact, so there the results have to be equal bit by bit.
"""
import pytest
import torch

import operator_cases as cases
import operator_refs as ref
from test_gpu_grouped import DT, check_all, moe, normal, operands  # noqa: F401 (moe is the fixture)

pytestmark = pytest.mark.gpu

SIZES = [(c, K, N, layout) for c, K, N, layout, *_ in cases.GROUPED]
each_size = pytest.mark.parametrize("counts,K,N,layout", SIZES)


def other(layout):
    return "kn" if layout == "nk" else "nk"


def name(counts, K, N, layout):
    return f"{counts if len(counts) < 9 else len(counts)} {K}x{N} {layout}"


@each_size
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_products_and_gradients(moe, counts, K, N, layout, dtype):  # noqa: F811
    check_all(moe, *operands(counts, K, N, layout, DT[dtype]), layout, name(counts, K, N, layout))


@each_size
def test_whole_numbers_are_exact(moe, counts, K, N, layout):  # noqa: F811
    print(name(counts, K, N, layout), flush=True)
    g = torch.Generator(device="cuda").manual_seed(3)

    def whole(*shape):
        return torch.randint(-1, 2, shape, generator=g, device="cuda").to(torch.bfloat16)

    R, E, off = sum(counts), len(counts), ref.offsets_of(counts)
    x, dy, w = whole(R, K), whole(R, N), whole(E, *((K, N) if layout == "kn" else (N, K)))
    y = moe.grouped_matmul(x, w, off, layout=layout)
    dx, dw = moe.grouped_matmul_backward(dy, x, w, off, layout=layout)
    a, b = (x, dy) if layout == "kn" else (dy, x)
    for got, want in ((y, ref.grouped(x, w, off, layout)[0]), (dx, ref.grouped(dy, w, off, other(layout))[0]), (dw, ref.grouped_dw(a, b, off)[0])):
        assert torch.equal(got, want.float().bfloat16())  # the sum is exact in 32 bits, and rounded once


@each_size
def test_rows_of_no_expert_give_zeros(moe, counts, K, N, layout):  # noqa: F811
    x, w, dy, off = operands(counts, K, N, layout, torch.bfloat16, before=5, after=140)
    for t in (x, dy):
        t[:5] = float("nan")
        t[5 + sum(counts):] = float("inf")
    check_all(moe, x, w, dy, off, layout, f"gaps {name(counts, K, N, layout)}")


@each_size
def test_nan_stays_with_its_expert(moe, counts, K, N, layout):  # noqa: F811
    print(name(counts, K, N, layout), flush=True)
    x, w, dy, off = operands(counts, K, N, layout, torch.float16)
    y = moe.grouped_matmul(x, w, off, layout=layout)
    dx, dw = moe.grouped_matmul_backward(dy, x, w, off, layout=layout)
    e = max(range(len(counts)), key=lambda i: counts[i])
    mine = torch.zeros(x.shape[0], dtype=torch.bool, device="cuda")
    mine[int(off[e]):int(off[e + 1])] = True
    x[mine] = dy[mine] = float("nan")
    y2 = moe.grouped_matmul(x, w, off, layout=layout)
    dx2, dw2 = moe.grouped_matmul_backward(dy, x, w, off, layout=layout)
    for a, b in ((y, y2), (dx, dx2)):
        assert torch.equal(a[~mine], b[~mine]) and bool(b[mine].isnan().all())
    rest = [i for i in range(len(counts)) if i != e]
    assert torch.equal(dw[rest], dw2[rest]) and bool(dw2[e].isnan().all())


@each_size
def test_one_nan_element_stays_in_its_row_and_column(moe, counts, K, N, layout):  # noqa: F811
    """The last element of a row and of a matrix, where tiles and steps are filled up."""
    print(name(counts, K, N, layout), flush=True)
    x, w, dy, off = operands(counts, K, N, layout, torch.bfloat16)
    y, dw = moe.grouped_matmul(x, w, off, layout=layout), moe.grouped_matmul_backward(dy, x, w, off, layout=layout, need_dx=False)[1]
    e = max(i for i in range(len(counts)) if counts[i])
    r = int(off[e + 1]) - 1
    x2, w2 = x.clone(), w.clone()
    x2[r, -1] = float("nan")
    got = moe.grouped_matmul(x2, w, off, layout=layout)
    assert bool(got[r].isnan().all())
    got[r] = y[r]
    assert torch.equal(got, y)
    got = moe.grouped_matmul_backward(dy, x2, w, off, layout=layout, need_dx=False)[1]
    hit = got[e][-1] if layout == "kn" else got[e][:, -1]
    assert bool(hit.isnan().all())
    hit.copy_(dw[e][-1] if layout == "kn" else dw[e][:, -1])
    assert torch.equal(got, dw)
    w2[e, -1, -1] = float("inf")
    got = moe.grouped_matmul(x, w2, off, layout=layout)
    rows = slice(int(off[e]), int(off[e + 1]))
    assert not bool(got[rows, -1].isfinite().any())
    got[rows, -1] = y[rows, -1]
    assert torch.equal(got, y)


@each_size
def test_replays_with_other_bounds(moe, counts, K, N, layout):  # noqa: F811
    print(name(counts, K, N, layout), flush=True)
    x, w, dy, off = operands(counts, K, N, layout, torch.bfloat16)
    R, E = sum(counts), len(counts)

    def step():
        return (moe.grouped_matmul(x, w, off, layout=layout),) + moe.grouped_matmul_backward(dy, x, w, off, layout=layout)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for i in range(4):
        g = torch.Generator().manual_seed(i)
        cuts = sorted(torch.randint(0, R + 1, (E + 1,), generator=g).tolist()) if i else [0] * E + [R]  # all to the last one first
        off.copy_(torch.tensor(cuts, dtype=torch.int32))
        x.copy_(normal(R, K, dtype=x.dtype, seed=20 + i))
        want = step()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(out, want):
            assert torch.equal(a, b), i
        ref.assert_within(want[0], *ref.grouped(x, w, off, layout), K, f"y after replay {i}")


def within_or_infinite(got, want, terms, n, what):
    """assert_within; a sum past the type's largest value by more than its bound has to be the infinity of its sign."""
    over = want.abs() - n * 2.0 ** -23 * terms >= torch.finfo(got.dtype).max * (1 + ref.HALF[got.dtype])
    assert bool((got[over].double() == want[over].sign() * float("inf")).all()), what
    ref.assert_within(torch.where(over, 0, got), torch.where(over, 0.0, want), terms, n, what)


@pytest.mark.parametrize("counts,K,N,layout", [s for s in SIZES if s[1] % 8 == 0 and s[2] % 8 == 0])
def test_rows_of_wider_tensors(moe, counts, K, N, layout):  # noqa: F811
    x, w, dy, off = operands(counts, K, N, layout, torch.float16)
    for lead in (8, 3):  # copied directly, and not
        big, wide = (normal(x.shape[0], n + 24, dtype=torch.float16, seed=9) for n in (K, N))
        big[:, lead:lead + K], wide[:, lead:lead + N] = x, dy
        check_all(moe, big[:, lead:lead + K], w, wide[:, lead:lead + N], off, layout, f"from column {lead}, {name(counts, K, N, layout)}")
    print("one row", flush=True)
    x, dy = x[:1].expand(x.shape[0], K), dy[:1].expand(x.shape[0], N)
    y = moe.grouped_matmul(x, w, off, layout=layout)
    dx, dw = moe.grouped_matmul_backward(dy, x, w, off, layout=layout)
    a, b = (x, dy) if layout == "kn" else (dy, x)
    within_or_infinite(y, *ref.grouped(x, w, off, layout), K, "y")
    within_or_infinite(dx, *ref.grouped(dy, w, off, other(layout)), N, "dx")
    within_or_infinite(dw, *ref.grouped_dw(a, b, off), max(counts), "dw")  # one product, thousands of times


GUARD = 4096


def guarded(rows, cols, dtype):
    """An output inside a buffer of a value that no result here has, and a check that the rest of it is untouched."""
    flat = torch.full((rows * cols + 2 * GUARD,), 777.0, dtype=dtype, device="cuda")

    def whole():
        return bool((flat[:GUARD] == 777).all()) and bool((flat[GUARD + rows * cols:] == 777).all())

    return flat[GUARD:GUARD + rows * cols].view(rows, cols), whole


def fits(got, want, terms, n):
    slack = n * 2.0 ** -23 * terms
    return (got.double() - want).abs() <= slack + ref.HALF[got.dtype] * (want.abs() + slack) + ref.TINY[got.dtype]


@each_size
def test_bounds_that_do_not_fit(moe, counts, K, N, layout):  # noqa: F811
    """Nothing outside an output is written; a row holds a product of an expert whose kept bounds have it, zeros if
    they are outside the first and last, or (where such rows overlap, and tiles are left over) what was there; the
    weights' gradients are those of the kept bounds."""
    import persistent_tile_scheduling_macro_amd as pg
    print(name(counts, K, N, layout), flush=True)
    x, w, dy, _ = operands(counts, K, N, layout, torch.bfloat16)
    R, E, nk = sum(counts), len(counts), layout == "nk"
    h = pg.pgemm_create(0)
    pg.pgemm_set_stream(h, torch.cuda.current_stream())
    products = [ref.grouped(x, w[e:e + 1], torch.tensor([0, R]), layout) for e in range(min(E, 5))]
    a, b = (dy, x) if nk else (x, dy)
    I, J = a.shape[1], b.shape[1]
    work = torch.zeros(max(16, pg.pgemm_grouped_weight_grad_workspace(R, E, I, J)), dtype=torch.uint8, device="cuda")
    top = 2 ** 31 - 1
    for bad in ([-7] + [R // 2] * (E - 1) + [top], [R - 3, 5] + [R] * (E - 1), [R] * E + [0], [top, -top - 1] * E, [0, R] * E):
        bad = bad[:E + 1]
        off = torch.tensor(bad, dtype=torch.int32, device="cuda")
        kept = [min(max(v, 0), R) for v in bad]
        spans = [(kept[e], max(kept[e], kept[e + 1])) for e in range(E)]
        outside = (kept[0], max(kept[0], kept[E]))
        y, intact = guarded(R, N, torch.bfloat16)
        pg.pgemm_grouped_run(h, x, K, w, off, y, R, E, K, N, int(nk), pg.PGEMM_BF16)
        torch.cuda.synchronize()
        assert intact(), bad
        row = torch.arange(R, device="cuda")[:, None]
        fine = (y == 0) & ((row < outside[0]) | (row >= outside[1]))
        cover = ((row < outside[0]) | (row >= outside[1])).long()
        checkable = torch.ones((R, 1), dtype=torch.bool, device="cuda")
        for e, (lo, hi) in enumerate(spans):
            inside = (row >= lo) & (row < hi)
            cover += inside
            if e < len(products):
                fine |= inside & fits(y, *products[e], K)
            else:
                checkable &= ~inside
        overlap = bool((cover > 1).any())
        if overlap:
            fine |= y == 777
        assert bool((fine | ~checkable).all()), bad
        c, intact = guarded(E * I, J, torch.bfloat16)
        pg.pgemm_grouped_weight_grad(h, a, I, b, J, off, c, R, E, I, J, pg.PGEMM_BF16, work, work.numel())
        torch.cuda.synchronize()
        assert intact(), bad
        for e, (lo, hi) in list(enumerate(spans))[:8]:
            want, terms = ref.grouped_dw(a[lo:hi], b[lo:hi], torch.tensor([0, hi - lo]))
            assert bool(fits(c.view(E, I, J)[e], want[0], terms[0], max(1, hi - lo)).all()), (bad, e)
    pg.pgemm_destroy(h)
