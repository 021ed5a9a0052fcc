"""GPU: how far the linear layer's gradients are from the definition's, and its largest gated sizes.

A rounding to 16 bits is off by a number spread evenly over one step, so its square has the mean step^2 / 12, and the errors
of different elements are independent. The gradients have three such roundings: z's as it is stored, which reaches dz through
the slope (gated: through both factors), dz's before the products (dbias adds up dz before it), and each gradient's own. The
squares of what they add to a product's output are the squares of dz's error times those of the other operand. All of that is
formed here in 64 bits; fp32's own errors are a hundredth of it.
"""
import pytest
import torch

import dense_cases as cases
import dense_refs as refs
from persistent_tile_scheduling_macro_amd import PGEMM_B_NK, pgemm_dense_query
from test_gpu_dense import check, dense, inputs  # noqa: F401  (a fixture)

pytestmark = pytest.mark.gpu


def variance(v, dtype):
    """Mean square error of rounding these values to dtype."""
    bits, least = {torch.float16: (10, -14), torch.bfloat16: (7, -126)}[dtype]
    exponent = torch.floor(torch.log2(v.abs().clamp(min=2.0 ** least)))
    return torch.exp2(exponent - bits) ** 2 / 12


def definition(dy, x, w, bias, name, gated):
    """(gradients, mean square error of each one's rounding path summed over its elements), layout nk, in 64 bits."""
    d, N, t = dy.double(), dy.shape[1], x.dtype
    z = x.double() @ w.double().t().contiguous() + bias.double()
    gate = z[:, :N]
    value, slope, _ = refs.act(name, gate)
    e = 1e-4
    bend = (refs.act(name, gate + e)[1] - refs.act(name, gate - e)[1]) / (2 * e)
    off = variance(gate, t) if gated or name != "none" else torch.zeros_like(gate)
    if gated:
        up = z[:, N:]
        dz = torch.cat([d * up * slope, d * value], 1)
        var = torch.cat([(d * up * bend) ** 2 * off + (d * slope) ** 2 * variance(up, t), (d * slope) ** 2 * off], 1)
    else:
        dz, var = d * slope, (d * bend) ** 2 * off
    grads = dz @ w.double(), dz.t().contiguous() @ x.double(), dz.sum(0)
    rounded = var + variance(dz, t) if gated or name != "none" else var  # dy itself, where it is dz, is not rounded again
    means = ((rounded @ (w.double() ** 2)).sum(), (rounded.t().contiguous() @ (x.double() ** 2)).sum(), var.sum())
    return grads, [m + variance(g, t).sum() for m, g in zip(means, grads)]


@pytest.mark.parametrize("M,N,K", [(120, 264, 200), (700, 520, 264), (2200, 1048, 520)])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("act,gated", [("none", False), ("gelu", False), ("gelu_tanh", False), ("silu", False), ("none", True),
                                       ("gelu", True), ("silu", True)])
def test_errors_of_the_gradients(dense, M, N, K, dtype, act, gated):  # noqa: F811
    x, w, b, _, dy = inputs(M, N, K, gated, "nk", dtype)
    _, z = dense.matmul(x, w, b, act=act, gated=gated, preactivation=True)
    got = dense.matmul_backward(dy, x, w, z, act=act, gated=gated, need_dbias=True)
    grads, means = definition(dy, x, w, b, act, gated)
    for g, want, mean, what in zip(got, grads, means, ("dx", "dw", "db")):
        error, expected = (g.double() - want).norm().item(), mean.sqrt().item()
        print(M, N, K, dtype, act, gated, what, "off by %.2e, %.2e expected" % (error / want.norm().item(), expected / want.norm().item()))
        # n independent errors: their sum of squares is off by some sqrt(2 / n) of itself, a dbias of 264 columns by a tenth
        assert error <= (1.1 if g.dim() == 2 else 1.3) * expected


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("act", ["gelu", "silu"])
@pytest.mark.parametrize("gated", [False, True])
def test_gradients_against_differences_in_any_direction(dense, dtype, act, gated):  # noqa: F811
    """The derivative along a random direction is off by one draw of the gradient's error: five times its size bounds it."""
    M, N, K = 40, 48, 64
    x, w, b, _, dy = inputs(M, N, K, gated, "nk", dtype, seed=3)
    _, z = dense.matmul(x, w, b, act=act, gated=gated, preactivation=True)
    grads = dense.matmul_backward(dy, x, w, z, act=act, gated=gated, need_dbias=True)
    _, means = definition(dy, x, w, b, act, gated)

    def loss(x, w, b):
        z = x @ w.t().contiguous() + b
        y = refs.act(act, z[:, :N])[0]
        return ((y * z[:, N:] if gated else y) * dy.double()).sum()

    at, h = [t.double() for t in (x, w, b)], 1e-5
    for i, g in enumerate(grads):
        for seed in range(4):
            d = torch.randn(at[i].shape, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda", dtype=torch.float64)
            plus, minus = list(at), list(at)
            plus[i], minus[i] = at[i] + h * d, at[i] - h * d
            numeric = (loss(*plus) - loss(*minus)) / (2 * h)
            assert abs((g.double() * d).sum() - numeric) <= 5 * means[i].sqrt()


@pytest.mark.parametrize("dtype,act", [("bf16", "silu"), ("f16", "gelu")])
def test_large_gated_gradients_are_read_past_the_cache(dense, dtype, act):  # noqa: F811
    """dy, gate and up of more bytes than the memory-side cache holds."""
    M, N = 8200, 4104
    assert N % 8 == 0 and 2 * M * (N + 2 * 2 * N) > 256 * 2 ** 20
    check(dense, M, N, 24, act, True, "nk", dtype, True, False)


@pytest.mark.parametrize("K,body", [(24, cases.PAIR), (520, cases.PING)])
def test_offsets_past_32_bits_in_aligned_gated_columns(dense, K, body):  # noqa: F811
    """More than 2^31 elements of z and dz, eight columns at a time: their last rows, and both halves' last columns."""
    M, N = 66001, 16504
    assert pgemm_dense_query(M, N, K, PGEMM_B_NK, 1) == (body, 1)
    x, w, _, _, dy = inputs(M, N, K, True, "nk", "bf16", False, False)
    y, z = dense.matmul(x, w, act="silu", gated=True, preactivation=True)
    assert z.numel() > 2 ** 31
    refs.check_forward(y[-70:], z[-70:], x[-70:], w, None, None, "silu", True, "nk")
    dx, dw, db = dense.matmul_backward(dy, x, w, z, act="silu", gated=True, need_dbias=True)
    refs.check_backward(dx[-70:], None, None, dy[-70:], x[-70:], w, z[-70:], "silu", True, "nk")

    def ends(t, dim):
        return torch.cat([t.narrow(dim, N - 8, 8), t.narrow(dim, 2 * N - 8, 8)], dim)

    refs.check_backward(None, ends(dw, 0), ends(db, 0), dy[:, -8:], x, ends(w, 0), ends(z, 1), "silu", True, "nk")
