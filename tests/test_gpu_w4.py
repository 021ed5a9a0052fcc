"""GPU: few rows times 4-bit weights against the plain form in 64 bits."""
import pytest
import torch

import operator_refs as ref

pytestmark = pytest.mark.gpu

DT = {"f16": torch.float16, "bf16": torch.bfloat16}
E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


@pytest.fixture(scope="module")
def w4():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from persistent_tile_scheduling_macro_amd import w4
    return w4


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def weights(N, K, group, dtype, zeros, E=0, seed=1):
    lead = (E,) if E else ()
    g, groups = gen(seed), -(-K // group)
    q = torch.randint(0, 256, lead + (N, (K + 1) // 2), generator=g, device="cuda", dtype=torch.uint8)
    s = ((torch.rand(lead + (N, groups), generator=g, device="cuda") + 0.1) * 0.02).to(dtype)
    z = torch.randint(0, 256, lead + (N, groups), generator=g, device="cuda", dtype=torch.uint8) if zeros else None
    return q, s, z


def values(q, s, z, K, group, fmt):
    """The weights in 64 bits."""
    code = torch.stack([q & 15, q >> 4], -1).flatten(-2)[..., :K].long()
    if fmt == "int4":
        zero = 8 if z is None else (z & 15).long().repeat_interleave(group, -1)[..., :K]
        v = (code - zero).double()
    else:
        v = torch.tensor(E2M1 + [-t for t in E2M1], dtype=torch.float64, device="cuda")[code]
    return v * s.double().repeat_interleave(group, -1)[..., :K]


def normal(*shape, dtype, seed):
    return torch.randn(shape, generator=gen(seed), device="cuda").to(dtype)


KINDS = [("int4", False), ("int4", True), ("e2m1", False)]


def check(w4, x, q, s, z, group, fmt, offsets=None, what=""):
    print(what, flush=True)
    K = x.shape[1]
    y = w4.matmul(x, q, s, z, group=group, fmt=fmt, offsets=offsets)
    w = values(q, s, z, K, group, fmt)
    # every product with a scale and every group's sum is one more step
    if offsets is None:
        xd = x.double()
        ref.assert_within(y, xd @ w.t().contiguous(), xd.abs() @ w.abs().t().contiguous(), 2 * K + 2, what)
    else:
        ref.assert_within(y, *ref.grouped(x, w, offsets, "nk"), 2 * K + 2, what)
    return y


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("fmt,zeros", KINDS)
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("M,N,K", [(1, 1, 1), (1, 64, 256), (3, 17, 129), (16, 48, 1000), (17, 70, 513), (33, 130, 2048),
                                   (64, 96, 640), (65, 33, 127), (130, 40, 1536), (2, 5000, 384), (5, 16, 31)])
def test_dense(w4, M, N, K, group, fmt, zeros, dtype):
    q, s, z = weights(N, K, group, DT[dtype], zeros)
    check(w4, normal(M, K, dtype=DT[dtype], seed=3), q, s, z, group, fmt, what=f"{M} {N} {K} {group} {fmt} {zeros} {dtype}")


@pytest.mark.parametrize("fmt,zeros", KINDS)
@pytest.mark.parametrize("counts,N,K", [([1], 32, 64), ([0, 3, 0, 1], 48, 300), ([20, 0, 17, 33], 70, 257), ([100, 2], 40, 1024), ([0, 0], 16, 64)])
def test_experts(w4, counts, N, K, fmt, zeros):
    for dtype in DT.values():
        q, s, z = weights(N, K, 64, dtype, zeros, len(counts))
        x = normal(sum(counts) + 3, K, dtype=dtype, seed=4)
        x[sum(counts):] = float("nan")  # rows of no expert
        off = ref.offsets_of(counts)
        y = check(w4, x, q, s, z, 64, fmt, off, f"{counts} {N} {K} {fmt}")
        assert not bool(y[sum(counts):].any())
        off = ref.offsets_of(counts, before=2)
        x = normal(sum(counts) + 2, K, dtype=dtype, seed=5)
        assert not bool(check(w4, x, q, s, z, 64, fmt, off, "gap in front")[:2].any())


def test_every_code_and_zero_point_is_exact(w4):
    """A one in x picks single weights: each code under each zero point, unrounded."""
    for dtype in DT.values():
        for fmt, zeros in KINDS:
            K, group = 512, 32
            code = torch.arange(K, device="cuda") % 16
            q = (code[0::2] | code[1::2] << 4).to(torch.uint8).repeat(16, 1)
            s = torch.tensor([0.25, 1.0, 2.0, 0.125], device="cuda").to(dtype).repeat(16, 4)
            z = (torch.arange(16, device="cuda", dtype=torch.uint8).repeat(16, 1)) if zeros else None
            x = torch.eye(K, device="cuda")[:48].to(dtype)
            y = w4.matmul(x, q, s, z, group=group, fmt=fmt)
            assert torch.equal(y.double(), values(q, s, z, K, group, fmt).t()[:48])


def test_strides_and_odd_addresses(w4):
    M, N, K, group = 9, 50, 520, 64
    for fmt, zeros in KINDS:
        q, s, z = weights(N, K, group, torch.bfloat16, zeros)
        wide = normal(M, K + 9, dtype=torch.bfloat16, seed=2)
        for lead in (0, 1, 8):
            check(w4, wide[:, lead:lead + K], q, s, z, group, fmt, what=f"slice at {lead}")
        check(w4, wide[:1, :K].expand(M, K), q, s, z, group, fmt, what="one row")

        def moved(t):
            flat = torch.empty(t.numel() + 1, dtype=t.dtype, device="cuda")
            flat[1:] = t.reshape(-1)
            return flat[1:].view(t.shape)

        check(w4, wide[:, :K], moved(q), moved(s), None if z is None else moved(z), group, fmt, what="odd addresses")
        check(w4, wide[:, :K], q.t().contiguous().t(), s.t().contiguous().t(), z, group, fmt, what="transposed")


def test_non_finite_rows_stay_in_their_rows(w4):
    q, s, _ = weights(40, 300, 32, torch.float16, False)
    x = normal(20, 300, dtype=torch.float16, seed=1)
    want = w4.matmul(x, q, s, group=32)
    x[7], x[19, 3] = float("nan"), float("inf")
    got = w4.matmul(x, q, s, group=32)
    keep = [i for i in range(20) if i not in (7, 19)]
    assert torch.equal(got[keep], want[keep]) and bool(got[7].isnan().all()) and not bool(got[19].isfinite().all())


def test_empty_sizes(w4):
    for M, N, K in ((0, 8, 64), (4, 0, 64), (4, 8, 0)):
        q, s, _ = weights(N, K, 64, torch.float16, False)
        y = w4.matmul(torch.ones((M, K), dtype=torch.float16, device="cuda"), q, s, group=64)
        assert y.shape == (M, N) and not bool(y.any())


def test_graph_replays_with_other_bounds(w4):
    q, s, z = weights(96, 384, 32, torch.bfloat16, True, 4)
    x, off = normal(24, 384, dtype=torch.bfloat16, seed=1), ref.offsets_of([6, 6, 6, 6])
    w4.matmul(x, q, s, z, group=32, offsets=off)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = w4.matmul(x, q, s, z, group=32, offsets=off)
    for i, counts in enumerate(([24, 0, 0, 0], [1, 2, 20, 1], [0, 0, 0, 0], [8, 0, 8, 7])):
        off.copy_(ref.offsets_of(counts))
        x.copy_(normal(24, 384, dtype=x.dtype, seed=10 + i))
        want = w4.matmul(x, q, s, z, group=32, offsets=off)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want), i


def test_another_stream(w4):
    q, s, _ = weights(512, 1024, 128, torch.float16, False)
    x = normal(4, 1024, dtype=torch.float16, seed=1)
    want = w4.matmul(x, q, s, group=128, fmt="e2m1")
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        got = w4.matmul(x * 1, q, s, group=128, fmt="e2m1")
    st.synchronize()
    assert torch.equal(got, want)


def test_weights_past_32_bit_offsets(w4):
    E, N, K = 36, 16384, 16384  # 4.8 GB of codes
    q = torch.zeros((E, N, K // 2), dtype=torch.uint8, device="cuda")
    s = torch.zeros((E, N, K // 128), dtype=torch.bfloat16, device="cuda")
    q1, s1, _ = weights(N, K, 128, torch.bfloat16, False)
    q[-1], s[-1] = q1, s1
    x = normal(3, K, dtype=torch.bfloat16, seed=2)
    off = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    off[-1] = 3
    assert torch.equal(w4.matmul(x, q, s, group=128, offsets=off), w4.matmul(x, q1, s1, group=128))


def test_bounds_that_do_not_fit_stay_inside(w4):
    q, s, _ = weights(48, 256, 32, torch.float16, False, 3)
    x = normal(20, 256, dtype=torch.float16, seed=1)
    for bad in ([0, 5, 900, 900], [-5, 3, 9, 12], [20, 9, 3, 0], [2147483647, 0, -2147483648, 20]):
        off = torch.tensor(bad, dtype=torch.int32, device="cuda")
        assert w4.matmul(x, q, s, group=32, offsets=off).shape == (20, 48)
        torch.cuda.synchronize()
