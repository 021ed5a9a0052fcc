"""Plain forms in 64 bits of the routed operators and the 4-bit product, and the bounds their tests hold them to.

A 16-bit output is one rounding of an fp32 sum. The rounding is off by at most half a step, eps/2 relative to the value
(plus half the smallest subnormal step); an fp32 sum of n terms, in any order, each step off by at most 2^-23 of what it
adds up (half a step to nearest, a whole one where the matrix unit truncates), by at most n * 2^-23 * sum|terms|.
"""
import torch

TINY = {torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -134, torch.float32: 2.0 ** -150}
HALF = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


def assert_within(got, want, terms, n, what=""):
    """got: rounded once to its type from an fp32 sum of n terms; want: the sum in 64 bits; terms: the sum of |terms|."""
    slack = n * 2.0 ** -23 * terms
    bound = slack + HALF[got.dtype] * (want.abs() + slack) + TINY[got.dtype]
    d = got.double() - want
    bad = ~(d.abs() <= bound)  # a NaN is bad too
    if bool(bad.any()):
        at = tuple(int(i) for i in torch.nonzero(bad)[0])
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} outside, first at {at}: "
                             f"{got[at].item()} for {want[at].item()}, bound {bound[at].item():.3g}")


def sort_slots(ids, E):
    """(offsets, order, pos) as int32: a stable sort of the kept slots by expert."""
    flat = ids.reshape(-1).cpu().tolist()
    kept = sorted((e, s) for s, e in enumerate(flat) if 0 <= e < E)
    order = [s for _, s in kept] + [-1] * (len(flat) - len(kept))
    pos = [-1] * len(flat)
    for p, (_, s) in enumerate(kept):
        pos[s] = p
    offsets = [0] * (E + 1)
    for e, _ in kept:
        offsets[e + 1] += 1
    for e in range(E):
        offsets[e + 1] += offsets[e]
    return tuple(torch.tensor(v, dtype=torch.int32, device=ids.device) for v in (offsets, order, pos))


def slot_rows(rows, pos, k):
    """The rows of every slot [T, k, H] in 64 bits, zeros for dropped ones (whatever any row holds)."""
    T = pos.numel() // k
    out = torch.zeros((pos.numel(), rows.shape[1]), dtype=torch.float64, device=rows.device)
    at = torch.nonzero(pos >= 0).reshape(-1)
    out[at] = rows[pos[at].long()].double()
    return out.view(T, k, -1)


def grouped(x, w, offsets, layout):
    """(y, sum of |terms|) in 64 bits."""
    off = offsets.tolist()
    N = w.shape[2] if layout == "kn" else w.shape[1]
    y = torch.zeros((x.shape[0], N), dtype=torch.float64, device=x.device)
    t = torch.zeros_like(y)
    for e in range(len(off) - 1):
        m = w[e].double() if layout == "kn" else w[e].double().t().contiguous()
        r = x[off[e]:off[e + 1]].double()
        y[off[e]:off[e + 1]] = r @ m
        t[off[e]:off[e + 1]] = r.abs() @ m.abs()
    return y, t


def grouped_dw(a, b, offsets):
    """(sum of a_r^T b_r over each expert's rows, sum of |terms|) in 64 bits."""
    off = offsets.tolist()
    E = len(off) - 1
    c = torch.zeros((E, a.shape[1], b.shape[1]), dtype=torch.float64, device=a.device)
    t = torch.zeros_like(c)
    for e in range(E):
        x, y = a[off[e]:off[e + 1]].double().t().contiguous(), b[off[e]:off[e + 1]].double()
        c[e], t[e] = x @ y, x.abs() @ y.abs()
    return c, t


def offsets_of(counts, before=0, device="cuda"):
    v = [before]
    for n in counts:
        v.append(v[-1] + n)
    return torch.tensor(v, dtype=torch.int32, device=device)
