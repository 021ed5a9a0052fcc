"""GPU: pre-activations beyond fp16's range, in the sums of every body. The forward pass has them in fp32; the copy that the
backward pass reads holds the type's largest value instead, so that no gradient is lost.
"""
import pytest
import torch

import dense_cases as cases
import dense_refs as refs
import operator_refs as ref

pytestmark = pytest.mark.gpu

MOST = 65504.0


@pytest.fixture(scope="module")
def dense():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from persistent_tile_scheduling_macro_amd import dense
    return dense


def one_of_each():
    """A size for every body, whole and in pieces, gated and not."""
    found = {}
    for M, N, K, layout, gated, (body, pieces) in cases.PRODUCTS:
        if layout == "nk" or (body, pieces > 1, gated) not in found:
            found[body, pieces > 1, gated] = M, N, K, layout, gated
    return sorted(found.values())


def inputs(M, N, K, layout, gated):
    """Rows 0, M / 2 and M - 1 have sums of 102400 and -102400 in two columns of the gate (of y) and, gated, in two of up."""
    g = torch.Generator(device="cuda").manual_seed(2)
    x = torch.randn((M, K), generator=g, device="cuda")
    w = torch.randn((N * (1 + gated), K), generator=g, device="cuda") * K ** -0.5
    x[:, 0], w[:, 0] = 0, 0
    x[[0, M // 2, M - 1], 0] = 256
    w[1, 0], w[N - 1, 0] = 400, -400
    if gated:
        w[N + 3, 0], w[2 * N - 4, 0] = 400, -400
    # gradients that the operands' type still holds after factors of 65504 and of 400 or 256, four and three of them added
    dy = torch.randn((M, N), generator=g, device="cuda").clamp(-2, 2) * 2.0 ** -12
    w = w.half() if layout == "nk" else w.half().t().contiguous()
    return x.half(), w, dy.half()


@pytest.mark.parametrize("act", refs.ACTS[1:])
@pytest.mark.parametrize("M,N,K,layout,gated", one_of_each())
def test_sums_beyond_fp16(dense, M, N, K, layout, gated, act):
    print(M, N, K, layout, gated, act, flush=True)
    x, w, dy = inputs(M, N, K, layout, gated)
    how = {"act": act, "gated": gated, "layout": layout}
    y, z = dense.matmul(x, w, preactivation=True, **how)
    xd, wd = refs.mats(x, w, layout)
    sums = xd @ wd
    far = sums.abs() > 1e5
    assert int(far.sum()) == 6 * (1 + gated)
    ref.assert_within(z, sums.clamp(-MOST, MOST), xd.abs() @ wd.abs(), K + 1, "z")
    assert torch.equal(z[far].double(), MOST * sums[far].sign())
    assert not bool(y.isnan().any()) and not bool(y[[0, M // 2, M - 1], N - 1].any())

    dx, dw, db = dense.matmul_backward(dy, x, w, z, need_dbias=True, **how)
    dz, err = refs.grad_of_z(dy, z, act, gated)
    # past 100 the activation is x or 0 and its slope 1 or 0, exactly: what rounds is the products with dy
    big = z[:, :N].double().abs() > 100
    big = torch.cat([big, big], 1) if gated else big
    err = torch.where(big, 2.0 ** -22 * dz.abs(), err)
    err = err + 2.0 ** -11 * (dz.abs() + err) + ref.TINY[torch.float16]
    reach = dz.abs() + err
    for got, want, e, terms, n, what in (
            (dx, dz @ wd.t(), err @ wd.abs().t(), reach @ wd.abs().t(), dz.shape[1], "dx"),
            (dw if layout == "kn" else dw.t(), xd.t() @ dz, xd.abs().t() @ err, xd.abs().t() @ reach, M, "dw"),
            (db, dz.sum(0), err.sum(0), reach.sum(0), M, "db")):
        e = e + n * 2.0 ** -23 * terms
        refs.outside(got, want, e + 2.0 ** -11 * (want.abs() + e) + ref.TINY[torch.float16], what)
    if not gated:  # the gradient by the sums themselves is the same: the slope there is 1 or 0 either way
        slope = refs.act(act, sums)[1]
        assert torch.equal((slope * dy.double())[far], dz[far])


@pytest.mark.parametrize("M", [3, 200])
@pytest.mark.parametrize("act", refs.ACTS[1:])
def test_infinite_and_nan_inputs_stay_what_they_are(dense, M, act):
    x = torch.ones((M, 64), device="cuda").half()
    x[0, 3], x[1, 5], x[2, 7] = float("inf"), float("-inf"), float("nan")
    _, z = dense.matmul(x, torch.ones((80, 64), device="cuda").half(), act=act, preactivation=True)
    assert bool((z[0] == float("inf")).all()) and bool((z[1] == float("-inf")).all()) and bool(z[2].isnan().all())
    assert bool((z[3:] == 64).all())
