"""CPU: the linear layer with its pre-activations returned records no gradient, and refuses what wants one."""
import pytest
import torch

from persistent_tile_scheduling_macro_amd import dense

SHAPES = {"x": (4, 8), "w": (6, 8), "bias": (6,), "residual": (4, 6)}


@pytest.mark.parametrize("which", SHAPES)
def test_preactivations_refuse_what_wants_a_gradient(which):
    args = {name: torch.zeros(shape, dtype=torch.float16) for name, shape in SHAPES.items()}
    args[which].requires_grad_(True)
    with pytest.raises(ValueError, match="no gradient"):
        dense.matmul(**args, act="silu", preactivation=True)
    with torch.no_grad(), pytest.raises(ValueError, match="on the GPU"):  # none is recorded: on to the next check
        dense.matmul(**args, act="silu", preactivation=True)
    args[which] = args[which].detach()
    with pytest.raises(ValueError, match="on the GPU"):
        dense.matmul(**args, act="silu", preactivation=True)
