"""GPU: what a token of the routed layer owes to the tokens beside it: nothing but the order in which its sums are added."""
import pytest
import torch

from test_gpu_layer import check, inputs, moe  # noqa: F401  (a fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,k,E,H,I,gated", [(8, 2, 40, 264, 1000, True), (33, 3, 50, 136, 517, False), (64, 2, 9, 520, 640, True)])
def test_a_token_among_others(moe, T, k, E, H, I, gated):  # noqa: F811
    x, ids, weights, w_in, w_out = inputs(T, k, E, H, I, gated, "bf16")
    out = moe.layer(x, ids, weights, w_in, w_out, gated=gated)
    for seed in (2, 3):
        other_x, other_ids, other_weights, _, _ = inputs(T, k, E, H, I, gated, "bf16", seed=seed)
        for t, mine in ((other_x, x), (other_ids, ids), (other_weights, weights)):
            t[T // 2] = mine[T // 2]
        # other rows and weights under the same ids: the same to the bit
        same = moe.layer(other_x, ids, torch.where(torch.arange(T, device="cuda")[:, None] == T // 2, weights, other_weights),
                         w_in, w_out, gated=gated)
        assert torch.equal(same[T // 2], out[T // 2])
        # other ids: as near the definition as before
        check(moe.layer(other_x, other_ids, other_weights, w_in, w_out, gated=gated), other_x, other_ids, other_weights, w_in, w_out,
              "silu", gated)
