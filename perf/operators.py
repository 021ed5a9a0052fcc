"""The routed operators and the 4-bit product: the cases they are measured on, and their plain forms.

Four operators. ``dispatch`` sorts token slots by expert and moves the rows; ``combine`` brings expert
outputs back to their tokens with the router's weights; ``grouped`` multiplies the sorted rows by their
expert's matrix; ``w4`` multiplies few rows by 4-bit weights with group scales, dense or per expert.
A case with ``train`` also returns the gradients.
"""
import torch

own = False  # True: run() calls the package's operators instead of the plain forms

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16}


def listed():
    return [
        # one serving step of a small batch: latency counts
        {"name": "dispatch step", "op": "dispatch", "T": 16, "k": 8, "E": 64, "H": 2048, "dtype": "bf16",
         "ids": "int32", "drop": 0.0, "skew": 0.0, "train": False},
        # a training batch of 8192 tokens, with the gradient of the rows
        {"name": "dispatch train", "op": "dispatch", "T": 8192, "k": 8, "E": 64, "H": 4096, "dtype": "bf16",
         "ids": "int64", "drop": 0.0, "skew": 0.1, "train": True},
        # a ragged prompt on one shard of the experts: some slots belong elsewhere and are dropped
        {"name": "dispatch ragged", "op": "dispatch", "T": 4099, "k": 2, "E": 13, "H": 1021, "dtype": "f16",
         "ids": "int64", "drop": 0.2, "skew": 0.5, "train": True},
        # the same three on the way back
        {"name": "combine step", "op": "combine", "T": 16, "k": 8, "E": 64, "H": 2048, "dtype": "bf16",
         "drop": 0.0, "skew": 0.0, "train": False},
        {"name": "combine train", "op": "combine", "T": 8192, "k": 8, "E": 64, "H": 4096, "dtype": "bf16",
         "drop": 0.0, "skew": 0.1, "train": True},
        {"name": "combine ragged", "op": "combine", "T": 4099, "k": 3, "E": 13, "H": 2056, "dtype": "f16",
         "drop": 0.2, "skew": 0.5, "train": True},
        # 32 tokens of a serving batch, 8 slots each: the experts' weights bound it
        {"name": "grouped few rows", "op": "grouped", "R": 256, "E": 32, "active": 32, "K": 2048, "N": 1536,
         "dtype": "bf16", "layout": "nk", "skew": 0.1, "train": False},
        # a training batch: 8192 tokens, 4 slots each, forward and both gradients
        {"name": "grouped train", "op": "grouped", "R": 32768, "E": 32, "active": 32, "K": 4096, "N": 2048,
         "dtype": "bf16", "layout": "kn", "skew": 0.1, "train": True},
        # ragged sizes, uneven experts, one of them empty
        {"name": "grouped ragged", "op": "grouped", "R": 8200, "E": 7, "active": 6, "K": 1000, "N": 2056,
         "dtype": "f16", "layout": "nk", "skew": 0.4, "train": True},
        # a single token through a square layer
        {"name": "w4 one row", "op": "w4", "M": 1, "E": 0, "active": 0, "N": 4096, "K": 4096, "group": 128,
         "fmt": "int4", "zeros": False, "dtype": "bf16"},
        # a full decoding batch through a wide layer, with zero points
        {"name": "w4 batch", "op": "w4", "M": 16, "E": 0, "active": 0, "N": 16384, "K": 8192, "group": 64,
         "fmt": "int4", "zeros": True, "dtype": "f16"},
        # three tokens of 8 slots over the experts' 4-bit weights
        {"name": "w4 experts", "op": "w4", "M": 24, "E": 32, "active": 16, "N": 2048, "K": 4096, "group": 32,
         "fmt": "e2m1", "zeros": False, "dtype": "bf16"},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(lo * (hi / lo) ** rng.random()))))


def _len(rng, lo, hi, odd=0.3):
    """A length, spread over the logarithm: a multiple of 8, or any number."""
    v = _log(rng, lo, hi)
    return v if rng.random() < odd else max(8, v // 8 * 8)


def draw(rng):
    op = rng.choice(["dispatch", "combine", "grouped", "w4"])
    dtype = rng.choice(["bf16", "f16"])
    if op in ("dispatch", "combine"):
        E = _log(rng, 2, 256)
        c = {"op": op, "T": _log(rng, 1, 8192), "k": rng.randint(1, min(8, E)), "E": E, "H": _len(rng, 64, 4096),
             "dtype": dtype, "drop": rng.choice([0.0, 0.0, 0.2]), "skew": rng.choice([0.0, 0.1, 0.5]),
             "train": rng.random() < 0.5}
        if op == "dispatch":
            c["ids"] = rng.choice(["int32", "int64"])
        return c
    if op == "grouped":
        E = _log(rng, 1, 64)
        K, N = _len(rng, 64, 4096), _len(rng, 64, 4096)
        R = min(_log(rng, 1, 32768), 32768 * 4096 * 2048 // (K * N))
        return {"op": op, "R": R, "E": E, "active": max(1, min(R, E - rng.choice([0, 0, 1]))), "K": K, "N": N,
                "dtype": dtype, "layout": rng.choice(["kn", "nk"]), "skew": rng.choice([0.0, 0.1, 0.4]),
                "train": rng.random() < 0.5}
    E = rng.choice([0, 0, _log(rng, 2, 32)])
    K = _len(rng, 256, 8192, 0.2)
    N = min(_len(rng, 64, 16384), 16384 * 8192 // (K * max(E, 1)))
    M = _log(rng, 1, 64)
    fmt = rng.choice(["int4", "int4", "e2m1"])
    return {"op": op, "M": M, "E": E, "active": min(M, rng.randint(1, E)) if E else 0, "N": N, "K": K,
            "group": rng.choice([32, 64, 128]), "fmt": fmt, "zeros": fmt == "int4" and rng.random() < 0.5,
            "dtype": dtype}


# ---------------------------------------------------------------- inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _ids(c, g):
    """k distinct experts for each token, some more popular than others; dropped slots name no expert."""
    T, k, E = c["T"], c["k"], c["E"]
    score = torch.rand((T, E), generator=g, device="cuda") + c["skew"] * torch.rand(E, generator=g, device="cuda")
    ids = score.topk(k, dim=1).indices
    away = torch.rand((T, k), generator=g, device="cuda") < c["drop"]
    return torch.where(away, torch.where(ids % 2 == 0, -1, E + 3), ids)


def _counts(rows, E, active, skew, g):
    """Rows of each expert: every active one has a row at least, the rest are dealt at random."""
    order = torch.randperm(E, generator=g, device="cuda")[:active]
    p = torch.exp(skew * torch.randn(active, generator=g, device="cuda"))
    n = torch.zeros(E, dtype=torch.int64, device="cuda")
    n[order] = 1
    if rows > active:
        n.index_add_(0, order[torch.multinomial(p, rows - active, replacement=True, generator=g)],
                     torch.ones(rows - active, dtype=torch.int64, device="cuda"))
    return n


def _offsets(counts):
    return torch.cat([torch.zeros(1, dtype=torch.int64, device="cuda"), counts.cumsum(0)]).to(torch.int32)


def _sorted(ids, E):
    """(offsets, order, pos) of the kept slots, sorted by expert, ties by slot."""
    n = ids.numel()
    key = torch.where((ids >= 0) & (ids < E), ids, E).reshape(-1).long()
    key, order = torch.sort(key, stable=True)
    at = torch.arange(n, device="cuda")
    kept = key < E
    offsets = torch.searchsorted(key, torch.arange(E + 1, device="cuda")).to(torch.int32)
    pos = torch.empty(n, dtype=torch.int32, device="cuda")
    pos[order] = torch.where(kept, at, -1).to(torch.int32)
    return offsets, torch.where(kept, order, -1).to(torch.int32), pos


def prepare(case, seed):
    c, g, dt = case, _gen(seed), DTYPES[case["dtype"]]
    s = {"case": dict(c)}

    def normal(*shape, scale=1.0):
        return (torch.randn(shape, generator=g, device="cuda", dtype=torch.float32) * scale).to(dt)

    if c["op"] == "dispatch":
        s["ids"] = _ids(c, g).to(torch.int32 if c["ids"] == "int32" else torch.int64)
        s["x"] = normal(c["T"], c["H"])
        if c["train"]:
            s["dxs"] = normal(c["T"] * c["k"], c["H"])
    elif c["op"] == "combine":
        s["offsets"], s["order"], s["pos"] = _sorted(_ids(c, g), c["E"])
        s["w"] = torch.softmax(torch.randn((c["T"], c["k"]), generator=g, device="cuda"), dim=1)
        s["ys"] = normal(c["T"] * c["k"], c["H"])
        if c["train"]:
            s["dout"] = normal(c["T"], c["H"])
    elif c["op"] == "grouped":
        counts = _counts(c["R"], c["E"], c["active"], c["skew"], g)
        s["offsets"], s["most"] = _offsets(counts), int(counts.max())
        s["x"] = normal(c["R"], c["K"])
        shape = (c["K"], c["N"]) if c["layout"] == "kn" else (c["N"], c["K"])
        s["w"] = normal(c["E"], *shape, scale=c["K"] ** -0.5)
        if c["train"]:
            s["dy"] = normal(c["R"], c["N"])
    else:
        E, N, K = c["E"], c["N"], c["K"]
        lead = (E,) if E else ()
        n_groups = -(-K // c["group"])
        s["x"] = normal(c["M"], K)
        s["q"] = torch.randint(0, 256, lead + (N, (K + 1) // 2), generator=g, device="cuda", dtype=torch.uint8)
        s["scales"] = (torch.rand(lead + (N, n_groups), generator=g, device="cuda") * 0.01 + 0.005).to(dt)
        s["zeros"] = (torch.randint(4, 12, lead + (N, n_groups), generator=g, device="cuda", dtype=torch.uint8)
                      if c["zeros"] else None)
        s["offsets"] = None
        if E:
            counts = _counts(c["M"], E, c["active"], 0.3, g)
            s["offsets"], s["most"] = _offsets(counts), int(counts.max())
    return s


# ------------------------------------------------------------ plain forms
def _plain_dispatch(s):
    c, x, ids = s["case"], s["x"], s["ids"]
    offsets, order, pos = _sorted(ids, c["E"])
    kept = (order >= 0)[:, None]
    xs = torch.where(kept, x[order.clamp(min=0).long() // c["k"]], 0)
    if not c["train"]:
        return offsets, order, pos, xs
    return offsets, order, pos, xs, _rows_back(s["dxs"], pos, c).sum(1).to(x.dtype)


def _rows_back(rows, pos, c):
    """Each slot's row in 32 bits, [T, k, H], zero for a dropped slot."""
    r = rows[pos.clamp(min=0).long()].float()
    return torch.where((pos >= 0)[:, None], r, 0.0).view(c["T"], c["k"], c["H"])


def _plain_combine(s):
    c, w = s["case"], s["w"]
    rows = _rows_back(s["ys"], s["pos"], c)
    out = (rows * w[:, :, None]).sum(1).to(s["ys"].dtype)
    if not c["train"]:
        return out
    dout = s["dout"].float()
    slot = s["order"].clamp(min=0).long()
    kept = (s["order"] >= 0)[:, None]
    dys = torch.where(kept, dout[slot // c["k"]] * w.reshape(-1)[slot][:, None], 0.0).to(s["ys"].dtype)
    dw = (rows * dout[:, None, :]).sum(2)
    return out, dys, dw


def _place(offsets, rows):
    """Expert and index within the expert of every sorted row."""
    at = torch.arange(rows, device="cuda", dtype=torch.int32)
    e = torch.searchsorted(offsets[1:], at, right=True)
    return e, (at - offsets[e]).long()


def _padded(x, e, i, E, most):
    p = torch.zeros((E, most, x.shape[1]), dtype=torch.float32, device="cuda")
    p[e, i] = x.float()
    return p


def _plain_grouped(s):
    c = s["case"]
    x, w = s["x"], s["w"].float()
    e, i = _place(s["offsets"], c["R"])
    xp = _padded(x, e, i, c["E"], s["most"])
    wkn = w if c["layout"] == "kn" else w.transpose(1, 2).contiguous()
    y = torch.bmm(xp, wkn)[e, i].to(x.dtype)
    if not c["train"]:
        return y
    dyp = _padded(s["dy"], e, i, c["E"], s["most"])
    wnk = w.transpose(1, 2).contiguous() if c["layout"] == "kn" else w
    dx = torch.bmm(dyp, wnk)[e, i].to(x.dtype)
    a, b = (xp, dyp) if c["layout"] == "kn" else (dyp, xp)
    dw = torch.bmm(a.transpose(1, 2).contiguous(), b).to(x.dtype)
    return y, dx, dw


E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _weights(s, dtype):
    """The 4-bit weights' values: low nibble first, each group with its scale and zero point."""
    c, q, K = s["case"], s["q"], s["case"]["K"]
    codes = torch.stack([q & 15, q >> 4], dim=-1).flatten(-2)[..., :K]
    if c["fmt"] == "int4":
        v = codes.to(dtype)
        z = 8.0 if s["zeros"] is None else s["zeros"].to(dtype).repeat_interleave(c["group"], -1)[..., :K]
        v = v - z
    else:
        table = torch.tensor(E2M1 + tuple(-t for t in E2M1), dtype=dtype, device="cuda")
        v = table[codes.int()]
    return v * s["scales"].to(dtype).repeat_interleave(c["group"], -1)[..., :K]


def _plain_w4(s):
    c, x = s["case"], s["x"]
    w = _weights(s, torch.float32)
    if not c["E"]:
        return (x.float() @ w.t()).to(x.dtype)
    e, i = _place(s["offsets"], c["M"])
    xp = _padded(x, e, i, c["E"], s["most"])
    return torch.bmm(xp, w.transpose(1, 2).contiguous())[e, i].to(x.dtype)


PLAIN = {"dispatch": _plain_dispatch, "combine": _plain_combine, "grouped": _plain_grouped, "w4": _plain_w4}


# ------------------------------------------------------ the package's calls
def _own(s):
    from persistent_tile_scheduling_macro_amd import moe, w4

    c = s["case"]
    if c["op"] == "dispatch":
        xs, plan = moe.dispatch(s["x"], s["ids"], c["E"])
        out = (plan.offsets, plan.order, plan.pos, xs)
        return out + (moe.dispatch_backward(s["dxs"], plan),) if c["train"] else out
    if c["op"] == "combine":
        plan = moe.RoutePlan(s["offsets"], s["order"], s["pos"], c["k"])
        out = moe.combine(s["ys"], s["w"], plan)
        return (out,) + tuple(moe.combine_backward(s["dout"], s["ys"], s["w"], plan)) if c["train"] else out
    if c["op"] == "grouped":
        y = moe.grouped_matmul(s["x"], s["w"], s["offsets"], layout=c["layout"])
        if not c["train"]:
            return y
        return (y,) + tuple(moe.grouped_matmul_backward(s["dy"], s["x"], s["w"], s["offsets"], layout=c["layout"]))
    return w4.matmul(s["x"], s["q"], s["scales"], s["zeros"], group=c["group"], fmt=c["fmt"], offsets=s["offsets"])


def run(state):
    return _own(state) if own else PLAIN[state["case"]["op"]](state)


# -------------------------------------------------------------------- work
def work(case):
    c = case
    if c["op"] in ("dispatch", "combine"):
        n, row = c["T"] * c["k"], 2 * c["H"]
        kept = int(n * (1 - c["drop"]))
        if c["op"] == "dispatch":
            b = n * (4 if c["ids"] == "int32" else 8) + 4 * (2 * n + c["E"] + 1) + c["T"] * row + n * row
            return {"bytes": b + c["train"] * (kept + c["T"]) * row, "flops": c["train"] * kept * c["H"]}
        b = 8 * n + kept * row + c["T"] * row
        return {"bytes": b + c["train"] * (c["T"] * row + n * row + 4 * n),
                "flops": 2 * kept * c["H"] + c["train"] * 3 * kept * c["H"]}
    if c["op"] == "grouped":
        R, K, N = c["R"], c["K"], c["N"]
        b = 2 * (R * K + R * N + c["active"] * K * N)
        return {"bytes": b + c["train"] * 2 * (R * N + R * K + c["E"] * K * N),
                "flops": (3 if c["train"] else 1) * 2 * R * K * N}
    M, N, K, n_w = c["M"], c["N"], c["K"], c["active"] or 1
    groups = -(-K // c["group"])
    return {"bytes": n_w * N * ((K + 1) // 2 + groups * (2 + c["zeros"])) + 2 * M * (K + N), "flops": 2 * M * N * K}


# ------------------------------------------------- the definitions in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    c = s["case"]
    if c["op"] == "dispatch":
        flat = s["ids"].reshape(-1).long()
        hot = flat[:, None] == torch.arange(c["E"], device="cuda")  # a slot's expert, one column each
        count = hot.sum(0)
        start = count.cumsum(0) - count
        rank = ((hot.cumsum(0) - 1 + start) * hot).sum(1)
        kept = hot.any(1)
        slots = torch.nonzero(kept).reshape(-1)
        n = flat.numel()
        pos = torch.where(kept, rank, -1)
        order = torch.full((n,), -1, dtype=torch.int64, device="cuda")
        order[rank[slots]] = slots
        xs = torch.zeros((n, c["H"]), dtype=torch.float64, device="cuda")
        xs[rank[slots]] = s["x"].double()[slots // c["k"]]
        offsets = torch.cat([start, count.sum()[None]])
        out = tuple(t.to(torch.int32) for t in (offsets, order, pos)) + (xs,)
        if not c["train"]:
            return out
        dx = torch.zeros((c["T"], c["H"]), dtype=torch.float64, device="cuda")
        for j in range(c["k"]):
            p = pos.view(c["T"], c["k"])[:, j]
            dx += torch.where((p >= 0)[:, None], s["dxs"][p.clamp(min=0)].double(), 0.0)
        return out + (dx,)
    if c["op"] == "combine":
        pos, w = s["pos"].view(c["T"], c["k"]).long(), s["w"].double()
        out = torch.zeros((c["T"], c["H"]), dtype=torch.float64, device="cuda")
        dys = torch.zeros((c["T"] * c["k"], c["H"]), dtype=torch.float64, device="cuda")
        dw = torch.zeros((c["T"], c["k"]), dtype=torch.float64, device="cuda")
        for j in range(c["k"]):
            t = torch.nonzero(pos[:, j] >= 0).reshape(-1)
            rows = s["ys"][pos[t, j]].double()
            out[t] += w[t, j, None] * rows
            if c["train"]:
                d = s["dout"][t].double()
                dys[pos[t, j]] = w[t, j, None] * d
                dw[t, j] = (rows * d).sum(1)
        return (out, dys, dw) if c["train"] else out
    if c["op"] == "grouped":
        off = s["offsets"].tolist()
        nk = c["layout"] == "nk"
        y = torch.zeros((c["R"], c["N"]), dtype=torch.float64, device="cuda")
        dx = torch.zeros((c["R"], c["K"]), dtype=torch.float64, device="cuda")
        dw = torch.zeros(s["w"].shape, dtype=torch.float64, device="cuda")
        for e in range(c["E"]):
            r = slice(off[e], off[e + 1])
            w, x = s["w"][e].double(), s["x"][r].double()
            y[r] = x @ (w.t() if nk else w)
            if c["train"]:
                d = s["dy"][r].double()
                dx[r] = d @ (w if nk else w.t())
                dw[e] = d.t() @ x if nk else x.t() @ d
        return (y, dx, dw) if c["train"] else y
    off = s["offsets"].tolist() if c["E"] else [0, c["M"]]
    y = torch.zeros((c["M"], c["N"]), dtype=torch.float64, device="cuda")
    for e in range(len(off) - 1):
        if off[e] == off[e + 1]:
            continue
        one = {"case": c, **{k: (s[k][e] if c["E"] and s[k] is not None else s[k]) for k in ("q", "scales", "zeros")}}
        lo, hi = one["q"] & 15, one["q"] >> 4
        code = torch.empty((c["N"], 2 * one["q"].shape[-1]), dtype=torch.int64, device="cuda")
        code[:, 0::2], code[:, 1::2] = lo.long(), hi.long()
        code = code[:, : c["K"]]
        group = torch.arange(c["K"], device="cuda") // c["group"]
        if c["fmt"] == "int4":
            v = (code - (8 if one["zeros"] is None else one["zeros"][:, group].long())).double()
        else:  # sign, two exponent bits, one mantissa bit
            ex, man = (code >> 1) & 3, code & 1
            v = torch.where(ex == 0, man * 0.5, (1 + man * 0.5) * torch.exp2(ex.double() - 1))
            v = torch.where(code >= 8, -v, v)
        y[off[e]: off[e + 1]] = s["x"][off[e]: off[e + 1]].double() @ (v * one["scales"][:, group].double()).t()
    return y
