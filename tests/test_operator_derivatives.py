"""CPU: derivatives that the routed operators and the 4-bit product do not record are refused, never dropped."""
import pytest
import torch
import torch.autograd.forward_ad as fwd

from persistent_tile_scheduling_macro_amd import moe, w4

F16, F32, U8, I32 = torch.float16, torch.float32, torch.uint8, torch.int32


def t(*shape, dtype=F16):
    return torch.zeros(shape, dtype=dtype)


def plan():
    return moe.RoutePlan(t(4, dtype=I32), t(8, dtype=I32), t(8, dtype=I32), 2)


# each call with its floating tensors, any one of which may carry the tangent
CALLS = [
    ([(4, 8, F16)], lambda x: moe.dispatch(x, t(4, 2, dtype=I32), 3)),
    ([(8, 8, F16)], lambda dxs: moe.dispatch_backward(dxs, plan())),
    ([(8, 8, F16), (4, 2, F32)], lambda ys, w: moe.combine(ys, w, plan())),
    ([(4, 8, F16), (8, 8, F16), (4, 2, F32)], lambda dout, ys, w: moe.combine_backward(dout, ys, w, plan())),
    ([(4, 8, F16), (2, 6, 8, F16)], lambda x, w: moe.grouped_matmul(x, w, t(3, dtype=I32))),
    ([(4, 6, F16), (4, 8, F16), (2, 6, 8, F16)], lambda dy, x, w: moe.grouped_matmul_backward(dy, x, w, t(3, dtype=I32))),
    ([(4, 64, F16), (8, 2, F16)], lambda x, s: w4.matmul(x, t(8, 32, dtype=U8), s, group=32)),
]
CASES = [(shapes, call, i) for shapes, call in CALLS for i in range(len(shapes))]


@pytest.mark.parametrize("shapes,call,which", CASES)
def test_tangents_are_refused(shapes, call, which):
    args = [t(*s[:-1], dtype=s[-1]) for s in shapes]
    with fwd.dual_level():
        args[which] = fwd.make_dual(args[which], torch.ones_like(args[which]))
        with pytest.raises(NotImplementedError, match="tangent"):
            call(*args)
        with torch.no_grad(), pytest.raises(NotImplementedError, match="tangent"):  # which is about reverse mode only
            call(*args)


def test_scales_that_want_a_gradient_are_refused():
    q, s = t(8, 32, dtype=U8), t(8, 2).requires_grad_(True)
    with pytest.raises(ValueError, match="no gradient"):
        w4.matmul(t(4, 64), q, s, group=32)
    with torch.no_grad(), pytest.raises(ValueError, match="on the GPU"):  # none is recorded: on to the next check
        w4.matmul(t(4, 64), q, s, group=32)


class HostDispatch:
    """The two bindings that moe.dispatch's autograd node calls, for one expert and two slots a token."""

    @staticmethod
    def dispatch(x, ids, E):
        n = 2 * x.shape[0]
        return x.repeat_interleave(2, 0), torch.tensor([0, n], dtype=I32), torch.arange(n, dtype=I32), torch.arange(n, dtype=I32)

    @staticmethod
    def dispatch_backward(dxs, offsets, order, pos, k):
        return dxs.view(-1, k, dxs.shape[1]).sum(1)


def test_a_plan_changed_before_the_backward_pass_is_noticed(monkeypatch):
    monkeypatch.setattr(moe, "_ops", HostDispatch)
    x = torch.ones(4, 8, dtype=F16, requires_grad=True)
    xs, route = moe.dispatch(x, t(4, 2, dtype=I32), 1)
    xs.sum().backward()
    assert torch.equal(x.grad, torch.full_like(x, 2))
    for name in ("offsets", "order", "pos"):
        xs, route = moe.dispatch(x, t(4, 2, dtype=I32), 1)
        getattr(route, name).fill_(0)
        with pytest.raises(RuntimeError, match="inplace"):
            xs.sum().backward()


def test_saved_tensor_hooks_see_the_plan(monkeypatch):
    monkeypatch.setattr(moe, "_ops", HostDispatch)
    x = torch.ones(4, 8, dtype=F16, requires_grad=True)
    packed = []
    with torch.autograd.graph.saved_tensors_hooks(lambda s: packed.append(s.shape) or s, lambda s: s):
        xs, _ = moe.dispatch(x, t(4, 2, dtype=I32), 1)
    assert sorted(packed) == [(2,), (8,), (8,)]
    xs.sum().backward()
