"""GPU: the 4-bit product in each form its rule chooses (rows at once, column blocks), against the plain form in 64 bits.

The sizes are those of operator_cases.py, which name their form; test_operator_coverage.py holds them to it on 256 CUs.
"""
import pytest
import torch

import operator_cases as cases
import operator_refs as ref
from test_gpu_w4 import DT, KINDS, check, gen, normal, values, weights, w4  # noqa: F401 (w4 is the fixture)

pytestmark = pytest.mark.gpu


def test_a_pass_stores_its_own_rows_only(w4):  # noqa: F811
    """Four rows at once and an expert of 14, in place in one workgroup: a pass that stored rows past its four would
    change what the next one reads."""
    import persistent_tile_scheduling_macro_amd as pg
    E, M, K = 8, 14, 16
    q, s, _ = weights(K, K, 32, torch.float16, False, E)
    x = normal(M, K, dtype=torch.float16, seed=1)
    off = torch.tensor([0, 0, 0, M, M, M, M, M, M], dtype=torch.int32, device="cuda")
    want = w4.matmul(x, q, s, group=32, offsets=off)
    ref.assert_within(want, *ref.grouped(x, values(q, s, None, K, 32, "int4"), off, "nk"), 2 * K + 2)
    h = pg.pgemm_create(0)
    pg.pgemm_set_stream(h, torch.cuda.current_stream())
    pg.pgemm_w4_run(h, x, K, q, s, None, off, x, M, K, K, E, 32, pg.PGEMM_W4_INT4, pg.PGEMM_F16)
    torch.cuda.synchronize()
    pg.pgemm_destroy(h)
    assert torch.equal(x, want)


def rows_of(E, M, seed):
    """Uneven rows of E experts, some without any."""
    share = torch.rand(E, generator=torch.Generator().manual_seed(seed)) ** 3
    share[::5] = 0
    counts = (share / share.sum() * M).long()
    counts[int(share.argmax())] += M - int(counts.sum())
    return counts.tolist()


@pytest.mark.parametrize("M,N,K,E,form", cases.W4)
@pytest.mark.parametrize("fmt,zeros", KINDS)
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_every_form(w4, M, N, K, E, form, group, fmt, zeros, dtype):  # noqa: F811
    import persistent_tile_scheduling_macro_amd as pg
    cus = torch.cuda.get_device_properties(0).multi_processor_count
    assert pg.pgemm_w4_query(M, N, E or 1, E > 0, cus) == form
    q, s, z = weights(N, K, group, DT[dtype], zeros, E)
    x = normal(M, K, dtype=DT[dtype], seed=3)
    off = ref.offsets_of(rows_of(E, M, 4)) if E else None
    check(w4, x, q, s, z, group, fmt, off, what=f"{M} {N} {K} {E} {form} {group} {fmt} {zeros} {dtype}")


# K of more steps than the scales a wave keeps at a time reach: read anew twice or three times
@pytest.mark.parametrize("group,K", [(32, 17011), (64, 33401), (128, 66000)])
@pytest.mark.parametrize("fmt,zeros", KINDS)
@pytest.mark.parametrize("M", [3, 16, 37])
@pytest.mark.parametrize("E", [0, 2])
def test_scales_are_read_anew_along_a_long_sum(w4, group, K, fmt, zeros, M, E):  # noqa: F811
    """Whole numbers and scales of a power of two: every sum is exact in 32 bits, so one wrong scale shows."""
    N = 40
    for dtype in DT.values():
        print(group, K, fmt, zeros, M, E, dtype, flush=True)
        q, _, z = weights(N, K, group, dtype, zeros, E)
        lead, g = ((E,) if E else ()), gen(8)
        s = torch.tensor([0.5, 1.0, 2.0, 4.0], device="cuda")[torch.randint(0, 4, lead + (N, -(-K // group)), generator=g, device="cuda")].to(dtype)
        x = torch.randint(-1, 2, (M, K), generator=g, device="cuda").to(dtype)
        off = ref.offsets_of([M - 2, 2]) if E else None
        y, w = w4.matmul(x, q, s, z, group=group, fmt=fmt, offsets=off), values(q, s, z, K, group, fmt)
        want = ref.grouped(x, w, off, "nk")[0] if E else x.double() @ w.t().contiguous()
        assert float(want.abs().max()) < 2 ** 16 - 32  # within fp16
        assert torch.equal(y, want.float().to(dtype))


GUARD = 4096


@pytest.mark.parametrize("M,N,K,E,form", [c for c in cases.W4 if c[3]])
def test_bounds_that_do_not_fit(w4, M, N, K, E, form):  # noqa: F811
    """Nothing outside y is written, and rows of one expert only, or of none, are right."""
    import persistent_tile_scheduling_macro_amd as pg
    h = pg.pgemm_create(0)
    pg.pgemm_set_stream(h, torch.cuda.current_stream())
    q, s, _ = weights(N, K, 32, torch.bfloat16, False, E)
    x = normal(M, K, dtype=torch.bfloat16, seed=1)
    w, top = values(q, s, None, K, 32, "int4"), 2 ** 31 - 1
    for bad in ([-7] + [M // 2] * (E - 1) + [top], [M - 3, 5] + [M] * (E - 1), [M] * E + [0], [top, -top - 1] * E, [0, M] * E):
        bad = bad[:E + 1]
        off = torch.tensor(bad, dtype=torch.int32, device="cuda")
        kept = [min(max(v, 0), M) for v in bad]
        flat = torch.full((M * N + 2 * GUARD,), 777.0, dtype=torch.bfloat16, device="cuda")
        y = flat[GUARD:GUARD + M * N].view(M, N)
        pg.pgemm_w4_run(h, x, K, q, s, None, off, y, M, N, K, E, 32, pg.PGEMM_W4_INT4, pg.PGEMM_BF16)
        torch.cuda.synchronize()
        assert bool((flat[:GUARD] == 777).all()) and bool((flat[GUARD + M * N:] == 777).all()), bad
        owners = [[] for _ in range(M)]
        for r in range(M):
            if r < kept[0] or r >= max(kept[0], kept[E]):
                owners[r].append(None)
            owners[r] += [e for e in range(E) if kept[e] <= r < max(kept[e], kept[e + 1])]
        for r in range(M):
            assert owners[r], (bad, r)
            if len(owners[r]) == 1:
                e = owners[r][0]
                m = w[e].t().contiguous() if e is not None else torch.zeros((K, N), dtype=torch.float64, device="cuda")
                xd = x[r:r + 1].double()
                ref.assert_within(y[r:r + 1], xd @ m, xd.abs() @ m.abs(), 2 * K + 2, f"{bad} row {r}")
    pg.pgemm_destroy(h)
