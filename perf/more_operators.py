"""The linear layer with its epilogue, the router and the routed layer of a few tokens: the cases they are measured
on, and their plain forms.

``dense`` multiplies rows by one matrix, adds a bias, applies an activation (or gates one half of the columns with the
other) and adds a residual; with ``train`` it also returns the pre-activations and all gradients. ``route`` chooses
each token's k experts from the router's logits and weighs them, with ``train`` also the logits' gradient. ``layer`` is
a whole mixture-of-experts layer for the few tokens of a decoding batch.
"""
import math

import torch

own = False  # True: run() calls the package's operators instead of the plain forms

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def listed():
    return [
        # one token through a square projection back into the residual stream: latency counts
        {"name": "dense token", "op": "dense", "M": 1, "K": 4096, "N": 4096, "dtype": "bf16", "layout": "nk",
         "act": "none", "gated": False, "bias": False, "residual": True, "train": False},
        # a decoding batch through a gated feed-forward layer's first matrix
        {"name": "dense step gated", "op": "dense", "M": 16, "K": 4096, "N": 8192, "dtype": "f16", "layout": "nk",
         "act": "silu", "gated": True, "bias": False, "residual": False, "train": False},
        # a short prompt
        {"name": "dense prompt", "op": "dense", "M": 512, "K": 8192, "N": 4096, "dtype": "bf16", "layout": "nk",
         "act": "gelu", "gated": False, "bias": True, "residual": True, "train": False},
        # a training batch of 8192 tokens, forward and all gradients
        {"name": "dense train", "op": "dense", "M": 8192, "K": 4096, "N": 8192, "dtype": "bf16", "layout": "nk",
         "act": "gelu_tanh", "gated": False, "bias": True, "residual": False, "train": True},
        # the gated form of it, the matrix stored by its input dimension
        {"name": "dense train gated", "op": "dense", "M": 4096, "K": 2048, "N": 4096, "dtype": "bf16", "layout": "kn",
         "act": "silu", "gated": True, "bias": False, "residual": False, "train": True},
        # odd sizes everywhere: a vocabulary-like width, a cropped batch
        {"name": "dense ragged", "op": "dense", "M": 4099, "K": 1021, "N": 2057, "dtype": "f16", "layout": "nk",
         "act": "gelu", "gated": False, "bias": True, "residual": True, "train": True},
        # the router of one decoding step
        {"name": "route step", "op": "route", "T": 16, "E": 64, "k": 8, "dtype": "bf16", "score": "softmax",
         "normalize": True, "masked": 0.0, "empty": 0.0, "train": False},
        # the router of a training batch with many experts
        {"name": "route train", "op": "route", "T": 8192, "E": 256, "k": 8, "dtype": "f32", "score": "softmax",
         "normalize": False, "masked": 0.0, "empty": 0.0, "train": True},
        # few experts, some of them closed to a token, some tokens padding
        {"name": "route ragged", "op": "route", "T": 4099, "E": 13, "k": 3, "dtype": "f16", "score": "sigmoid",
         "normalize": True, "masked": 0.4, "empty": 0.1, "train": True},
        # one token through eight of 64 experts
        {"name": "layer token", "op": "layer", "T": 1, "k": 8, "E": 64, "H": 2048, "I": 1024, "dtype": "bf16",
         "act": "silu", "gated": True, "drop": 0.0},
        # a decoding batch that wakes nearly every expert
        {"name": "layer batch", "op": "layer", "T": 32, "k": 4, "E": 32, "H": 4096, "I": 2048, "dtype": "bf16",
         "act": "silu", "gated": True, "drop": 0.0},
        # odd sizes on one shard of the experts: some slots belong elsewhere
        {"name": "layer ragged", "op": "layer", "T": 11, "k": 3, "E": 13, "H": 1021, "I": 517, "dtype": "f16",
         "act": "gelu", "gated": False, "drop": 0.2},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(lo * (hi / lo) ** rng.random()))))


def _len(rng, lo, hi, odd=0.3):
    """A length, spread over the logarithm: a multiple of 8, or any number."""
    v = _log(rng, lo, hi)
    return v if rng.random() < odd else max(8, v // 8 * 8)


def draw(rng):
    op = rng.choice(["dense", "dense", "dense", "route", "layer", "layer"])
    if op == "dense":
        K, N, gated = _len(rng, 64, 8192), _len(rng, 64, 8192), rng.random() < 0.4
        M = max(1, min(_log(rng, 1, 8192), 8192 * 4096 * 8192 // (K * N * (1 + gated))))
        train = rng.random() < 0.5
        # relu's slope jumps at zero, where the order of a sum decides its sign: forward only
        acts = ["gelu", "gelu_tanh", "silu"] + ([] if gated else ["none"]) + ([] if train else ["relu"])
        return {"op": op, "M": M, "K": K, "N": N, "dtype": rng.choice(["bf16", "f16"]),
                "layout": rng.choice(["nk", "nk", "kn"]), "act": rng.choice(acts), "gated": gated,
                "bias": rng.random() < 0.5, "residual": rng.random() < 0.5, "train": train}
    if op == "route":
        E = _log(rng, 2, 512)
        return {"op": op, "T": _log(rng, 1, 8192), "E": E, "k": rng.randint(1, min(8, E)),
                "dtype": rng.choice(["f32", "bf16", "f16"]), "score": rng.choice(["softmax", "softmax", "sigmoid"]),
                "normalize": rng.random() < 0.5, "masked": rng.choice([0.0, 0.3]), "empty": rng.choice([0.0, 0.1]),
                "train": rng.random() < 0.5}
    E = _log(rng, 2, 128)
    H, I = _len(rng, 256, 4096), _len(rng, 128, 4096)
    E = max(2, min(E, 32 * 4096 * 2048 // (H * I)))
    return {"op": op, "T": _log(rng, 1, 64), "k": rng.randint(1, min(8, E)), "E": E, "H": H, "I": I,
            "dtype": rng.choice(["bf16", "f16"]), "act": rng.choice(["silu", "silu", "gelu", "gelu_tanh", "relu"]),
            "gated": rng.random() < 0.7, "drop": rng.choice([0.0, 0.0, 0.2])}


# ---------------------------------------------------------------- inputs
def prepare(case, seed):
    c, dt = case, DTYPES[case["dtype"]]
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    s = {"case": dict(c)}

    def normal(*shape, scale=1.0, dtype=dt):
        return (torch.randn(shape, generator=g, device="cuda", dtype=torch.float32) * scale).to(dtype)

    if c["op"] == "dense":
        M, K, N, columns = c["M"], c["K"], c["N"], c["N"] * (1 + c["gated"])
        s["x"] = normal(M, K)
        s["w"] = normal(*((columns, K) if c["layout"] == "nk" else (K, columns)), scale=K ** -0.5)
        s["bias"] = normal(columns, scale=0.5) if c["bias"] else None
        s["residual"] = normal(M, N) if c["residual"] else None
        if c["train"]:
            s["dy"] = normal(M, N)
    elif c["op"] == "route":
        T, E = c["T"], c["E"]
        logits = torch.randn((T, E), generator=g, device="cuda") * 1.5
        closed = torch.rand((T, E), generator=g, device="cuda") < c["masked"]
        closed |= torch.rand((T, 1), generator=g, device="cuda") < c["empty"]
        s["logits"] = logits.masked_fill(closed, -math.inf).to(dt)
        if c["train"]:
            s["dweights"] = normal(T, c["k"], dtype=torch.float32)
    else:
        T, k, E, H, I = c["T"], c["k"], c["E"], c["H"], c["I"]
        s["x"] = normal(T, H)
        ids = torch.rand((T, E), generator=g, device="cuda").topk(k, dim=1).indices
        away = torch.rand((T, k), generator=g, device="cuda") < c["drop"]
        s["ids"] = torch.where(away, -1, ids).to(torch.int32)
        s["weights"] = torch.softmax(torch.randn((T, k), generator=g, device="cuda"), dim=1)
        s["w_in"] = normal(E, I * (1 + c["gated"]), H, scale=H ** -0.5)
        s["w_out"] = normal(E, H, I, scale=I ** -0.5)
    return s


# ------------------------------------------------------------ plain forms
_TANH_A, _TANH_B = math.sqrt(2 / math.pi), 0.044715


def _act(name, v):
    if name == "relu":
        return torch.clamp(v, min=0)
    if name == "gelu":
        return v * 0.5 * (1 + torch.erf(v * math.sqrt(0.5)))
    if name == "gelu_tanh":
        return 0.5 * v * (1 + torch.tanh(_TANH_A * (v + _TANH_B * v * v * v)))
    if name == "silu":
        return v / (1 + torch.exp(-v))
    return v


def _act_slope(name, v):
    if name == "relu":
        return (v > 0).to(v.dtype)
    if name == "gelu":
        return 0.5 * (1 + torch.erf(v * math.sqrt(0.5))) + v * torch.exp(-0.5 * v * v) * (1 / math.sqrt(2 * math.pi))
    if name == "gelu_tanh":
        t = torch.tanh(_TANH_A * (v + _TANH_B * v * v * v))
        return 0.5 * (1 + t) + 0.5 * v * (1 - t * t) * _TANH_A * (1 + 3 * _TANH_B * v * v)
    if name == "silu":
        p = 1 / (1 + torch.exp(-v))
        return p * (1 + v * (1 - p))
    return torch.ones_like(v)


def _plain_dense(s):
    c, x, w = s["case"], s["x"].float(), s["w"].float()
    nk, dt, N = c["layout"] == "nk", s["x"].dtype, c["N"]
    z = x @ (w.t() if nk else w)
    if c["bias"]:
        z = z + s["bias"].float()
    y = _act(c["act"], z[:, :N]) * z[:, N:] if c["gated"] else _act(c["act"], z)
    if c["residual"]:
        y = y + s["residual"].float()
    if not c["train"]:
        return y.to(dt)
    dy = s["dy"].float()
    if c["gated"]:
        dz = torch.cat([dy * z[:, N:] * _act_slope(c["act"], z[:, :N]), dy * _act(c["act"], z[:, :N])], dim=1)
    else:
        dz = dy * _act_slope(c["act"], z)
    dx = dz @ (w if nk else w.t())
    dw = dz.t() @ x if nk else x.t() @ dz
    out = {"y": y.to(dt), "dx": dx.to(dt), "dw": dw.to(dt)}
    if c["act"] != "none":
        out["z"] = z.to(dt)
    if c["bias"]:
        out["db"] = dz.sum(0).to(dt)
    return out


def _plain_route(s):
    c, logits = s["case"], s["logits"].float()
    top, ids = torch.sort(logits, dim=1, descending=True, stable=True)
    top, ids = top[:, :c["k"]], ids[:, :c["k"]]
    live = top > -math.inf
    if c["score"] == "softmax":
        most = torch.where(live[:, :1], top[:, :1], 0.0)
        part = torch.exp(top - most)
        every = torch.exp(logits - most)
    else:
        part = 1 / (1 + torch.exp(-top))
        every = None
    if c["normalize"]:
        total = part.sum(1, keepdim=True)
    else:
        total = every.sum(1, keepdim=True) if c["score"] == "softmax" else torch.ones_like(part)
    weights = torch.where(live, part / total, 0.0)
    chosen = torch.where(live, ids, -1).to(torch.int32)
    if not c["train"]:
        return chosen, weights
    dw = torch.where(live, s["dweights"], 0.0)
    mean = (weights * dw).sum(1, keepdim=True)
    if c["score"] == "softmax":
        grad = torch.zeros_like(logits).scatter_(1, ids, weights * (dw - mean if c["normalize"] else dw))
        if not c["normalize"]:
            grad = grad - torch.where(live[:, :1], every / total * mean, 0.0)
    else:
        slope = (dw - mean) / total if c["normalize"] else dw
        grad = torch.zeros_like(logits).scatter_(1, ids, torch.where(live, slope * part * (1 - part), 0.0))
    return chosen, weights, grad.to(s["logits"].dtype)


def _plain_layer(s):
    c, x, I = s["case"], s["x"].float(), s["case"]["I"]
    out = torch.zeros((c["T"], c["H"]), dtype=torch.float32, device="cuda")
    for e in range(c["E"]):
        share = torch.where(s["ids"] == e, s["weights"], 0.0).sum(1, keepdim=True)
        z = x @ s["w_in"][e].float().t()
        h = _act(c["act"], z[:, :I]) * z[:, I:] if c["gated"] else _act(c["act"], z)
        out += share * (h @ s["w_out"][e].float().t())
    return out.to(s["x"].dtype)


PLAIN = {"dense": _plain_dense, "route": _plain_route, "layer": _plain_layer}


# ------------------------------------------------------ the package's calls
def _own(s):
    from persistent_tile_scheduling_macro_amd import dense, moe

    c = s["case"]
    if c["op"] == "dense":
        how = {"act": c["act"], "gated": c["gated"], "layout": c["layout"]}
        if not c["train"]:
            return dense.matmul(s["x"], s["w"], s["bias"], s["residual"], **how)
        y, z = dense.matmul(s["x"], s["w"], s["bias"], s["residual"], preactivation=True, **how)
        dx, dw, db = dense.matmul_backward(s["dy"], s["x"], s["w"], z, need_dbias=c["bias"], **how)
        out = {"y": y, "dx": dx, "dw": dw}
        if z is not None:
            out["z"] = z
        if c["bias"]:
            out["db"] = db
        return out
    if c["op"] == "route":
        how = {"score": c["score"], "normalize": c["normalize"]}
        ids, weights = moe.route(s["logits"], c["k"], **how)
        if not c["train"]:
            return ids, weights
        return ids, weights, moe.route_backward(s["dweights"], s["logits"], ids, weights, **how)
    return moe.layer(s["x"], s["ids"], s["weights"], s["w_in"], s["w_out"], act=c["act"], gated=c["gated"])


def run(state):
    return _own(state) if own else PLAIN[state["case"]["op"]](state)


# -------------------------------------------------------------------- work
def work(case):
    c = case
    if c["op"] == "dense":
        M, K, N, cols = c["M"], c["K"], c["N"], c["N"] * (1 + c["gated"])
        kept = M * cols * (c["act"] != "none")  # the pre-activations, where a gradient needs them
        b = M * K + K * cols + M * N + c["residual"] * M * N + c["bias"] * cols
        if c["train"]:  # dy in, pre-activations, dx, dw, db out
            b += M * N + kept + M * K + K * cols + c["bias"] * cols
        return {"bytes": 2 * b, "flops": (3 if c["train"] else 1) * 2 * M * K * cols}
    if c["op"] == "route":
        T, E, k, size = c["T"], c["E"], c["k"], 4 if c["dtype"] == "f32" else 2
        b = T * E * size + 8 * T * k
        return {"bytes": b + c["train"] * (T * E * size + 4 * T * k), "flops": 8 * T * E * (1 + c["train"])}
    T, k, E, H, I = c["T"], c["k"], c["E"], c["H"], c["I"]
    matrix = H * I * (2 + c["gated"])
    taken = k / E * (1 - c["drop"])
    awake = E * (1 - (1 - taken) ** T)  # experts that some token takes, on average
    return {"bytes": int(2 * awake * matrix + 4 * T * H + 8 * T * k), "flops": int(2 * T * k * (1 - c["drop"]) * matrix)}


# ------------------------------------------------- the definitions in 64 bits
def _phi(v):
    return torch.special.ndtr(v)


def _exact_act(name, v):
    """(value, slope) of the activation."""
    if name == "none":
        return v, torch.ones_like(v)
    if name == "relu":
        up = (v > 0).double()
        return v * up, up
    if name == "gelu":
        return v * _phi(v), _phi(v) + v * torch.exp(-v.square() / 2) / math.sqrt(2 * math.pi)
    if name == "silu":
        p = torch.sigmoid(v)
        return v * p, p + v * p * (1 - p)
    u = math.sqrt(8 / math.pi) * (v + 0.044715 * v ** 3)  # (1 + tanh(u / 2)) / 2 = sigmoid(u)
    p = torch.sigmoid(u)
    return v * p, p + v * p * (1 - p) * math.sqrt(8 / math.pi) * (1 + 0.134145 * v ** 2)


def exact(case, seed):
    s = prepare(case, seed)
    c = s["case"]
    if c["op"] == "dense":
        x, w, N = s["x"].double(), s["w"].double(), c["N"]
        if c["layout"] == "nk":
            w = w.t()  # [K, columns] from here on
        z = torch.mm(x, w)
        if c["bias"]:
            z += s["bias"].double()
        value, slope = _exact_act(c["act"], z[:, :N])
        y = value * z[:, N:] if c["gated"] else value
        if c["residual"]:
            y = y + s["residual"].double()
        if not c["train"]:
            return y
        dy = s["dy"].double()
        dz = torch.empty_like(z)
        dz[:, :N] = dy * slope * (z[:, N:] if c["gated"] else 1.0)
        if c["gated"]:
            dz[:, N:] = dy * value
        dw = torch.mm(x.t(), dz)
        out = {"y": y, "dx": torch.mm(dz, w.t()), "dw": dw.t() if c["layout"] == "nk" else dw}
        if c["act"] != "none":
            out["z"] = z
        if c["bias"]:
            out["db"] = dz.sum(0)
        return out
    if c["op"] == "route":
        l, k = s["logits"].double(), c["k"]
        left = l.clone()
        ids, live, rows = [], [], torch.arange(c["T"], device="cuda")
        for _ in range(k):  # the largest that is left, the first of equals
            best = left.max(1).values
            at = (left == best[:, None]).double().argmax(1)
            live.append(best > -math.inf)
            ids.append(at)
            left[rows, at] = -math.inf
        ids, live = torch.stack(ids, 1), torch.stack(live, 1)
        # scores as a full matrix, then the chosen entries of it
        hot = torch.zeros_like(l)
        for j in range(k):
            hot[rows, ids[:, j]] = torch.where(live[:, j], 1.0, hot[rows, ids[:, j]])
        if c["score"] == "softmax":
            score = torch.exp(l - torch.logsumexp(l, 1, keepdim=True).nan_to_num(neginf=0.0))
        else:
            score = torch.sigmoid(l)
        total = (score * hot).sum(1, keepdim=True)
        share = torch.where(hot > 0, score / total, 0.0) if c["normalize"] else score * hot
        weights = torch.where(live, share.gather(1, ids), 0.0)
        chosen = torch.where(live, ids, -1).to(torch.int32)
        if not c["train"]:
            return chosen, weights
        d = torch.zeros_like(l)
        for j in range(k):
            d[rows, ids[:, j]] += torch.where(live[:, j], s["dweights"][:, j].double(), 0.0)
        if c["normalize"]:  # through share = score / total
            d = torch.where(hot > 0, (d - (d * share).sum(1, keepdim=True)) / total, 0.0)
        if c["score"] == "softmax":
            return chosen, weights, score * (d - (d * score).sum(1, keepdim=True))
        return chosen, weights, d * score * (1 - score)
    out = torch.zeros((c["T"], c["H"]), dtype=torch.float64, device="cuda")
    for t, row in enumerate(s["ids"].tolist()):
        for j, e in enumerate(row):
            if 0 <= e < c["E"]:
                z = s["w_in"][e].double() @ s["x"][t].double()
                value, _ = _exact_act(c["act"], z[:c["I"]])
                h = value * z[c["I"]:] if c["gated"] else value
                out[t] += s["weights"][t, j].double() * (s["w_out"][e].double() @ h)
    return out
