"""A mixture-of-experts layer: one training step in bf16, then decoding with its weights in four bits.

    python examples/moe_layer.py

Training: the router's choices send each token's row to its experts (moe.dispatch), two grouped products with a gated
activation between them, and the rows come back weighted (moe.combine); gradients run through the same operators.
Decoding: the trained matrices, as int4 codes with a scale for every 64 elements, multiply a few rows (w4.matmul).
"""
import os
import sys

import torch
import torch.nn.functional as F

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from persistent_tile_scheduling_macro_amd import moe, w4  # noqa: E402

GROUP = 64


def route(x, router, k):
    """Each token's k experts and their weights, which sum to one."""
    weights, ids = torch.topk(torch.softmax(x.float() @ router, dim=1), k, dim=1)
    return ids, weights / weights.sum(1, keepdim=True)


def layer(x, router, w_in, w_out, k, product):
    """x [T, H] through the experts; product(rows, w, offsets) multiplies sorted rows by their expert's matrix."""
    ids, weights = route(x, router, k)
    rows, plan = moe.dispatch(x, ids, router.shape[1])
    gate, up = product(rows, w_in, plan.offsets).chunk(2, dim=1)
    return moe.combine(product(F.silu(gate) * up, w_out, plan.offsets), weights, plan)


def quantize(w):
    """int4 codes [E, N, K/2], scales and zero points [E, N, K/GROUP] of w [E, N, K]; K a multiple of GROUP."""
    g = w.float().unflatten(-1, (-1, GROUP))
    low, high = g.amin(-1).clamp(max=0), g.amax(-1).clamp(min=0)
    scale = ((high - low) / 15).clamp(min=1e-8).to(w.dtype)
    zero = (-low / scale.float()).round().clamp(0, 15)
    code = (g / scale.float()[..., None] + zero[..., None]).round().clamp(0, 15).to(torch.uint8).flatten(-2)
    return code[..., 0::2] | code[..., 1::2] << 4, scale, zero.to(torch.uint8)


def run(T=512, H=256, W=384, E=8, k=2, steps=3, device="cuda:0"):
    """Trains the layer towards a fixed target; returns the losses and how far the 4-bit decode is from the bf16 one."""
    torch.manual_seed(0)

    def leaf(*shape, fan, dtype=torch.bfloat16):
        return (torch.randn(shape, device=device) * fan ** -0.5).to(dtype).requires_grad_(True)

    router = leaf(H, E, fan=H, dtype=torch.float32)
    w_in, w_out = leaf(E, 2 * W, H, fan=H), leaf(E, H, W, fan=W)
    x = torch.randn(T, H, device=device).bfloat16()
    target = torch.randn(T, H, device=device)
    optimizer = torch.optim.SGD([router, w_in, w_out], lr=50.0)
    losses = []
    for _ in range(steps):
        out = layer(x, router, w_in, w_out, k, lambda r, w, o: moe.grouped_matmul(r, w, o, layout="nk"))
        loss = F.mse_loss(out.float(), target)
        optimizer.zero_grad()
        loss.backward()
        optimizer.step()
        losses.append(loss.item())

    with torch.no_grad():
        few = x[:4]
        want = layer(few, router, w_in, w_out, k, lambda r, w, o: moe.grouped_matmul(r, w, o, layout="nk"))
        packed = {id(w): quantize(w) for w in (w_in, w_out)}
        got = layer(few, router, w_in, w_out, k,
                    lambda r, w, o: w4.matmul(r, *packed[id(w)], group=GROUP, offsets=o))
        off = ((got - want).float().norm() / want.float().norm()).item()
    return losses, off


if __name__ == "__main__":
    losses, off = run()
    print("loss of each step:", " ".join(f"{v:.4f}" for v in losses))
    print(f"4-bit decode against bf16: relative difference {off:.3f}")
