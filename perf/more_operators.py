"""Cases that time the operators which train an expert layer around dispatch and combine, in bf16.

Six operators; rows are grouped by expert as the dispatch lays them out (expert_offsets, slot_row):

  router         the experts of each token and their weights from the router's logits, and the logits' gradient
  combine_grad   gradient of the weighted sum over a token's experts: of the expert rows and of the weights
  dispatch_grad  gradient of the dispatch: a token's expert rows added up, on top of what other paths brought
  linear         the experts' product (or one dense product) with bias, activation and residual
  input_grad     gradient of the product by its rows, times the derivative of the activation in front of it
  weight_grad    gradient of the product by its weights and bias

``run`` computes them in elementary torch operations in 32 bits, or, with ``own`` set, calls the package.
"""
import math

import torch

own = False


# ---- the cases -----------------------------------------------------------------

def listed():
    return [
        # one sequence's new token in front of an expert layer, chosen by biased sigmoid scores: latency
        {"name": "router_token", "op": "router", "T": 1, "E": 256, "topk": 8, "score": "sigmoid", "bias": True,
         "normalize": True, "scale": 2.5, "logits": "f32", "train": False},
        # a training step's tokens, 64 ranks of 256: choice and gradient, every logit has one
        {"name": "router_train", "op": "router", "T": 16384, "E": 384, "topk": 8, "score": "softmax", "bias": False,
         "normalize": False, "scale": 1.0, "logits": "f32", "train": True},
        # the smallest layer: latency
        {"name": "combine_grad_tiny", "op": "combine_grad", "T": 64, "H": 256, "topk": 2, "E": 8, "skew": 0.0},
        # 32 ranks of 128 tokens over 256 experts: the memory's case
        {"name": "combine_grad_experts", "op": "combine_grad", "T": 4096, "H": 7168, "topk": 8, "E": 256, "skew": 0.0},
        # an odd batch with odd rows, on top of the gradient that the skip path and the router brought
        {"name": "dispatch_grad_odd", "op": "dispatch_grad", "T": 1001, "H": 1416, "topk": 3, "E": 40, "skew": 0.5,
         "add": True},
        # 64 ranks of 256 tokens under a skewed router
        {"name": "dispatch_grad_experts", "op": "dispatch_grad", "T": 16384, "H": 7168, "topk": 8, "E": 384,
         "skew": 1.0, "add": False},
        # a dense layer for one new token, residual added: all the weights are read for one row
        {"name": "linear_token", "op": "linear", "T": 1, "topk": 1, "E": 1, "N": 7168, "K": 2048, "skew": 0.0,
         "activation": "gelu", "bias": "bf16", "residual": True, "pre": False, "out": "bf16"},
        # gate and up of 256 experts over 32 ranks of 128 tokens, what the gradient needs kept
        {"name": "linear_experts", "op": "linear", "T": 4096, "topk": 8, "E": 256, "N": 2048, "K": 7168, "skew": 0.0,
         "activation": "swiglu", "bias": "", "residual": False, "pre": True, "out": "bf16"},
        # ragged groups under a skewed router, odd sizes in all three directions
        {"name": "input_grad_ragged", "op": "input_grad", "T": 1001, "topk": 3, "E": 40, "N": 1416, "K": 2320,
         "skew": 1.0, "activation": "gelu", "out": "bf16"},
        # through the second product and the gate of eight experts, a thousand rows each: the tensor cores' case
        {"name": "input_grad_experts", "op": "input_grad", "T": 4096, "topk": 2, "E": 8, "N": 4096, "K": 8192,
         "skew": 0.0, "activation": "swiglu", "out": "bf16"},
        # ragged groups, some without a row, float32 gradients
        {"name": "weight_grad_ragged", "op": "weight_grad", "T": 333, "topk": 2, "E": 40, "N": 1416, "K": 840,
         "skew": 1.0, "bias": True, "out": "f32"},
        # the first product of eight experts, a thousand rows each
        {"name": "weight_grad_experts", "op": "weight_grad", "T": 4096, "topk": 2, "E": 8, "N": 16384, "K": 4096,
         "skew": 0.0, "bias": False, "out": "bf16"},
    ]


def _spread(rng, lo, hi, step=1):
    """A size between lo and hi, spread over its logarithm, a multiple of step."""
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi))) / step)) * step
    return min(max(v, step, lo), hi // step * step)


def draw(rng):
    op = rng.choice(["router", "combine_grad", "dispatch_grad", "linear", "input_grad", "weight_grad"])
    while True:
        if op == "router":
            E = _spread(rng, 2, 1024)
            score = rng.choice(["softmax", "sigmoid"])
            c = {"op": op, "T": _spread(rng, 1, 16384), "E": E, "topk": min(E, rng.randint(1, 16)), "score": score,
                 "bias": score == "sigmoid" and rng.random() < 0.6, "normalize": rng.random() < 0.6,
                 "scale": rng.choice([1.0, 2.5]), "logits": rng.choice(["f32", "bf16"]), "train": rng.random() < 0.6}
            if c["T"] * E <= 16384 * 384:
                return c
            continue
        grouped = op in ("combine_grad", "dispatch_grad") or rng.random() < 0.6
        E = _spread(rng, 2, 384) if grouped else 1
        c = {"op": op, "T": _spread(rng, 1, 16384), "topk": min(E, rng.randint(1, 8)), "E": E,
             "skew": rng.choice([0.0, 0.5, 1.0]) if grouped else 0.0}
        if op in ("combine_grad", "dispatch_grad"):
            c["H"] = _spread(rng, 64, 7168, 8)
            if op == "dispatch_grad":
                c["add"] = rng.random() < 0.5
            return c
        c.update(N=_spread(rng, 128, 8192, 16), K=_spread(rng, 128, 8192, 8), out=rng.choice(["bf16", "f32"]))
        if op == "linear":
            c["activation"] = rng.choice(["none", "relu", "gelu", "silu", "swiglu"])
            c.update(bias=rng.choice(["", "bf16", "f32"]), residual=rng.random() < 0.4, pre=rng.random() < 0.5)
        elif op == "input_grad":
            c.update(activation=rng.choice(["none", "relu", "gelu", "silu", "swiglu"]), out="bf16")
        else:
            c["bias"] = rng.random() < 0.5
        if E * c["N"] * c["K"] <= 1.8e9 and work(c)["flops"] <= 8e11:
            return c


def _experts_with_rows(T, topk, E):
    """How many of E experts T tokens reach, on average, with topk different ones each."""
    return E * (1.0 - (1.0 - topk / E) ** T)


def work(case):
    c = case
    T, topk, E, op = c["T"], c["topk"], c["E"], c["op"]
    rows = T * topk
    if op == "router":
        size = 4 if c["logits"] == "f32" else 2
        back = rows * 4 + T * E * size if c["train"] else 0
        return {"bytes": T * E * size + rows * 8 + (4 * E if c["bias"] else 0) + back,
                "flops": T * E * (12 if c["train"] else 6)}
    if op == "combine_grad":
        return {"bytes": (T + 2 * rows) * c["H"] * 2 + rows * 12, "flops": 3 * rows * c["H"]}
    if op == "dispatch_grad":
        return {"bytes": (rows + T * (2 if c["add"] else 1)) * c["H"] * 2 + rows * 4, "flops": rows * c["H"]}
    N, K = c["N"], c["K"]
    active = min(_experts_with_rows(T, topk, E), E)
    size = 2 if c["out"] == "bf16" else 4
    if op == "linear":
        n_out = N // 2 if c["activation"] == "swiglu" else N
        per_expert = N * K * 2 + N * {"": 0, "bf16": 2, "f32": 4}[c["bias"]]
        per_row = K * 2 + n_out * size + (n_out * 2 if c["residual"] else 0) + (N * 2 if c["pre"] else 0)
    elif op == "input_grad":
        wide = 2 if c["activation"] == "swiglu" else 1
        per_expert = N * K * 2
        per_row = N * 2 + wide * K * 2 + (0 if c["activation"] == "none" else wide * K * 2)
    else:
        active = E  # the gradient of an expert without rows is written too
        per_expert = N * K * size + (N * 4 if c["bias"] else 0)
        per_row = (N + K) * 2
    return {"bytes": active * per_expert + rows * per_row, "flops": 2 * rows * N * K}


# ---- the inputs -----------------------------------------------------------------

def _type(name):
    return torch.bfloat16 if name == "bf16" else torch.float32


def _rows(g, rows, n, size=1.0):
    """Activations or gradients: normal values, a few channels larger, rows of different size."""
    v = torch.randn(rows, n, generator=g, device="cuda")
    v *= size * torch.exp(0.5 * torch.randn(rows, 1, generator=g, device="cuda"))
    v[:, :: max(1, n // 4)] *= 4.0
    return v.to(torch.bfloat16)


def _choices(g, T, topk, E, skew):
    """topk different experts for each token and their weights, popularity spread by skew."""
    popularity = skew * torch.randn(1, E, generator=g, device="cuda")
    u = torch.rand(T, E, generator=g, device="cuda").clamp_(1e-7, 1.0 - 1e-7)
    score, idx = torch.topk(popularity - torch.log(-torch.log(u)), topk, dim=1)
    return idx.to(torch.int32), torch.softmax(score, 1)


def _dispatched(s, idx, E):
    """What a dispatch of these choices leaves in its layout."""
    flat = idx.flatten().long()
    order = torch.argsort(flat, stable=True)
    slot_row = torch.empty_like(flat)
    slot_row[order] = torch.arange(flat.numel(), device=flat.device)
    s["slot_row"] = slot_row.view(idx.shape).to(torch.int32)
    counts = torch.bincount(flat, minlength=E)
    s["offsets"] = torch.cat([torch.zeros_like(counts[:1]), counts.cumsum(0)]).to(torch.int32)


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    s = {"case": c}
    bf16 = dict(dtype=torch.bfloat16, device="cuda")
    f32 = dict(dtype=torch.float32, device="cuda")
    op, T, topk, E = c["op"], c["T"], c["topk"], c["E"]
    rows = T * topk
    if op == "router":
        s["logits"] = (1.5 * torch.randn(T, E, generator=g, device="cuda")).to(_type(c["logits"]))
        s["bias"] = 0.1 * torch.randn(E, generator=g, device="cuda") if c["bias"] else None
        s["dw"] = torch.randn(T, topk, generator=g, device="cuda") if c["train"] else None
        s["idx"] = torch.empty(T, topk, dtype=torch.int32, device="cuda")
        s["w"] = torch.empty(T, topk, **f32)
        s["d_logits"] = torch.empty_like(s["logits"]) if c["train"] else None
        return s
    idx, weights = _choices(g, T, topk, E, c["skew"])
    if op in ("combine_grad", "dispatch_grad"):
        H = c["H"]
        _dispatched(s, idx, E)
        s["expert_rows"] = _rows(g, rows, H)
        if op == "combine_grad":
            s["weights"] = weights
            s["d_out"] = _rows(g, T, H, 0.1)
            s["d_expert_rows"] = torch.empty(rows, H, **bf16)
            s["d_weights"] = torch.empty(T, topk, **f32)
        else:
            s["add"] = _rows(g, T, H) if c["add"] else None
            s["dx"] = torch.empty(T, H, **bf16)
        return s
    if E > 1:
        _dispatched(s, idx, E)
        s["bounds"] = s["offsets"].tolist()  # the plain form's: it takes one expert after the other
    else:
        s["offsets"], s["bounds"] = None, [0, rows]
    N, K = c["N"], c["K"]
    if op == "weight_grad":
        s["dy"] = _rows(g, rows, N, 0.1)
        s["a"] = _rows(g, rows, K)
        s["dw"] = torch.empty(E, N, K, dtype=_type(c["out"]), device="cuda")
        s["db"] = torch.empty(E, N, **f32) if c["bias"] else None
        return s
    s["w"] = torch.randn(E, N, K, generator=g, **bf16).mul_(1.0 / math.sqrt(K if op == "linear" else N))
    if op == "linear":
        n_out = N // 2 if c["activation"] == "swiglu" else N
        s["a"] = _rows(g, rows, K)
        s["bias"] = torch.randn(E, N, generator=g, device="cuda").to(_type(c["bias"])) if c["bias"] else None
        s["residual"] = _rows(g, rows, n_out) if c["residual"] else None
        s["pre"] = torch.empty(rows, N, **bf16) if c["pre"] else None
        s["out"] = torch.empty(rows, n_out, dtype=_type(c["out"]), device="cuda")
    else:
        wide = 2 * K if c["activation"] == "swiglu" else K
        s["dy"] = _rows(g, rows, N, 0.1)
        s["pre"] = None if c["activation"] == "none" else _rows(g, rows, wide)
        s["dx"] = torch.empty(rows, wide, **bf16)
    return s


# ---- one pass -------------------------------------------------------------------

def _scores(logits, score):
    if score == "sigmoid":
        return 1.0 / (1.0 + torch.exp(-logits))
    p = torch.exp(logits - logits.amax(1, keepdim=True))
    return p / p.sum(1, keepdim=True)


def _plain_router(s):
    c = s["case"]
    # The choice in 64 bits: of two scores next to each other the larger one is taken.
    key = s["logits"].double()
    if c["bias"]:
        key = _scores(key, "sigmoid") + s["bias"].double()
    idx = torch.sort(key, dim=1, descending=True, stable=True)[1][:, : c["topk"]]
    p = _scores(s["logits"].float(), c["score"])
    chosen = p.gather(1, idx)
    total = chosen.sum(1, keepdim=True)
    share = chosen / total if c["normalize"] else chosen
    out = {"idx": idx.to(torch.int32), "w": c["scale"] * share}
    if c["train"]:
        dp = c["scale"] * s["dw"]
        if c["normalize"]:
            dp = (dp - (dp * share).sum(1, keepdim=True)) / total
        full = torch.zeros_like(p).scatter_(1, idx, dp)
        if c["score"] == "sigmoid":
            d = full * p * (1.0 - p)
        else:
            d = p * (full - (full * p).sum(1, keepdim=True))
        out["d_logits"] = d.to(s["logits"].dtype)
    return out


def _activation(name, v):
    if name == "relu":
        return v.clamp_min(0.0)
    if name == "gelu":
        return 0.5 * v * (1.0 + torch.erf(v * math.sqrt(0.5)))
    if name == "silu":
        return v / (1.0 + torch.exp(-v))
    if name == "swiglu":
        gate, up = v.chunk(2, 1)
        return gate / (1.0 + torch.exp(-gate)) * up
    return v


def _through_activation(name, v, d):
    """d times the derivative of the activation at v."""
    if name == "relu":
        return d * (v > 0.0).to(d.dtype)
    if name == "gelu":
        density = torch.exp(-0.5 * v * v) * (1.0 / math.sqrt(2.0 * math.pi))
        return d * (0.5 * (1.0 + torch.erf(v * math.sqrt(0.5))) + v * density)
    if name == "silu":
        sig = 1.0 / (1.0 + torch.exp(-v))
        return d * sig * (1.0 + v * (1.0 - sig))
    if name == "swiglu":
        gate, up = v.chunk(2, 1)
        sig = 1.0 / (1.0 + torch.exp(-gate))
        return torch.cat([d * up * sig * (1.0 + gate * (1.0 - sig)), d * gate * sig], 1)
    return d


def _plain(s):
    c = s["case"]
    op = c["op"]
    if op == "router":
        return _plain_router(s)
    if op == "combine_grad":
        at = s["slot_row"].flatten().long()
        token = torch.arange(at.numel(), device=at.device) // c["topk"]
        d_out = s["d_out"].float()[token]
        dy = torch.empty_like(s["expert_rows"])
        dy[at] = (s["weights"].flatten()[:, None] * d_out).to(dy.dtype)
        dw = (d_out * s["expert_rows"].float()[at]).sum(1)
        return {"d_expert_rows": dy, "d_weights": dw.view(s["weights"].shape)}
    if op == "dispatch_grad":
        dx = s["expert_rows"].float()[s["slot_row"].long()].sum(1)
        if c["add"]:
            dx = dx + s["add"].float()
        return {"dx": dx.to(torch.bfloat16)}
    groups = list(zip(s["bounds"][:-1], s["bounds"][1:]))
    if op == "linear":
        out = torch.empty_like(s["out"])
        pre = torch.empty_like(s["pre"]) if c["pre"] else None
        for e, (lo, hi) in enumerate(groups):
            if hi == lo:
                continue
            v = s["a"][lo:hi].float() @ s["w"][e].float().t()
            if c["bias"]:
                v = v + s["bias"][e].float()
            if c["pre"]:
                pre[lo:hi] = v.to(pre.dtype)
            v = _activation(c["activation"], v)
            if c["residual"]:
                v = v + s["residual"][lo:hi].float()
            out[lo:hi] = v.to(out.dtype)
        return {"out": out, "pre": pre} if c["pre"] else {"out": out}
    if op == "input_grad":
        dx = torch.empty_like(s["dx"])
        for e, (lo, hi) in enumerate(groups):
            if hi > lo:
                d = s["dy"][lo:hi].float() @ s["w"][e].float()
                v = None if s["pre"] is None else s["pre"][lo:hi].float()
                dx[lo:hi] = _through_activation(c["activation"], v, d).to(dx.dtype)
        return {"dx": dx}
    dw = torch.empty_like(s["dw"])
    db = torch.empty_like(s["db"]) if c["bias"] else None
    for e, (lo, hi) in enumerate(groups):
        dy = s["dy"][lo:hi].float()
        dw[e] = (dy.t() @ s["a"][lo:hi].float()).to(dw.dtype)
        if c["bias"]:
            db[e] = dy.sum(0)
    return {"dw": dw, "db": db} if c["bias"] else {"dw": dw}


def _own(s):
    from combine_route_count_gb300 import train
    c = s["case"]
    op = c["op"]
    if op == "router":
        train.router_topk(s["logits"], s["idx"], s["w"], score=c["score"], bias=s["bias"], normalize=c["normalize"],
                          scale=c["scale"])
        out = {"idx": s["idx"], "w": s["w"]}
        if c["train"]:
            train.router_topk_backward(s["logits"], s["idx"], s["dw"], s["d_logits"], score=c["score"],
                                       normalize=c["normalize"], scale=c["scale"])
            out["d_logits"] = s["d_logits"]
        return out
    if op == "combine_grad":
        train.combine_backward(s["d_out"], s["slot_row"], s["weights"], s["d_expert_rows"], expert_y=s["expert_rows"],
                               d_topk_w=s["d_weights"])
        return {"d_expert_rows": s["d_expert_rows"], "d_weights": s["d_weights"]}
    if op == "dispatch_grad":
        train.dispatch_backward(s["expert_rows"], s["slot_row"], s["dx"], add=s["add"])
        return {"dx": s["dx"]}
    if op == "linear":
        train.expert_linear(s["a"], s["w"], s["out"], bias=s["bias"], activation=c["activation"],
                            residual=s["residual"], pre=s["pre"], expert_offsets=s["offsets"])
        return {"out": s["out"], "pre": s["pre"]} if c["pre"] else {"out": s["out"]}
    if op == "input_grad":
        train.expert_linear_backward_input(s["dy"], s["w"], s["dx"], activation=c["activation"], pre=s["pre"],
                                           expert_offsets=s["offsets"])
        return {"dx": s["dx"]}
    train.expert_linear_backward_weight(s["dy"], s["a"], s["dw"], db=s["db"], expert_offsets=s["offsets"])
    return {"dw": s["dw"], "db": s["db"]} if c["bias"] else {"dw": s["dw"]}


def run(state):
    return _own(state) if own else _plain(state)


# ---- the definition in 64 bits ---------------------------------------------------

def _exact_router(s):
    c = s["case"]
    z = s["logits"].double()
    sig = torch.sigmoid(z)
    key = sig + s["bias"].double() if c["bias"] else z
    # The largest first, the lowest index among equals: one choice after the other.
    idx = torch.empty(c["T"], c["topk"], dtype=torch.int64, device=z.device)
    left, lane = key.clone(), torch.arange(c["E"], device=z.device)
    for k in range(c["topk"]):
        best = left == left.amax(1, keepdim=True)
        idx[:, k] = torch.where(best, lane, c["E"]).amin(1)
        left.scatter_(1, idx[:, k : k + 1], -math.inf)
    log_score = torch.nn.functional.logsigmoid(z) if c["score"] == "sigmoid" else torch.log_softmax(z, 1)
    log_chosen = log_score.gather(1, idx)
    w = torch.softmax(log_chosen, 1) if c["normalize"] else log_chosen.exp()
    out = {"idx": idx.to(torch.int32), "w": c["scale"] * w}
    if c["train"]:
        dw = c["scale"] * s["dw"].double()
        # By the logarithms of the chosen scores, then by the logits.
        d_log = w * (dw - (dw * w).sum(1, keepdim=True)) if c["normalize"] else w * dw
        d = torch.zeros_like(z).scatter_(1, idx, d_log)
        if c["score"] == "sigmoid":
            d *= torch.sigmoid(-z)
        else:
            d -= torch.softmax(z, 1) * d_log.sum(1, keepdim=True)
        out["d_logits"] = d
    return out


def _phi(v):
    return 0.5 * torch.erfc(-v / math.sqrt(2.0))


def _forward64(name, v):
    if name == "relu":
        return torch.where(v > 0, v, torch.zeros_like(v))
    if name == "gelu":
        return v * _phi(v)
    if name == "silu":
        return v * torch.sigmoid(v)
    if name == "swiglu":
        n = v.shape[1] // 2
        return v[:, :n] * torch.sigmoid(v[:, :n]) * v[:, n:]
    return v


def _slope64(name, v):
    if name == "relu":
        return torch.where(v > 0, torch.ones_like(v), torch.zeros_like(v))
    if name == "gelu":
        return _phi(v) + v * torch.exp(-v * v / 2) / math.sqrt(2 * math.pi)
    return torch.sigmoid(v) + v * torch.sigmoid(v) * torch.sigmoid(-v)  # silu


def exact(case, seed):
    if work(case)["flops"] > 4e12:
        return None
    s, c = prepare(case, seed), case
    op = c["op"]
    if op == "router":
        return _exact_router(s)
    f64 = dict(dtype=torch.float64, device="cuda")
    if op == "combine_grad":
        dy = torch.empty(s["expert_rows"].shape, **f64)
        dw = torch.empty(s["weights"].shape, **f64)
        for k in range(c["topk"]):
            at = s["slot_row"][:, k].long()
            dy[at] = s["weights"][:, k].double()[:, None] * s["d_out"].double()
            dw[:, k] = torch.einsum("th,th->t", s["d_out"].double(), s["expert_rows"][at].double())
        return {"d_expert_rows": dy, "d_weights": dw}
    if op == "dispatch_grad":
        dx = s["add"].double() if c["add"] else torch.zeros(c["T"], c["H"], **f64)
        for k in range(c["topk"]):
            dx += s["expert_rows"][s["slot_row"][:, k].long()].double()
        return {"dx": dx}
    off = [0, c["T"] * c["topk"]] if s["offsets"] is None else s["offsets"].tolist()
    if op == "linear":
        pre = torch.empty(off[-1], c["N"], **f64)
        for e in range(c["E"]):
            lo, hi = off[e], off[e + 1]
            if hi > lo:
                torch.mm(s["a"][lo:hi].double(), s["w"][e].double().t(), out=pre[lo:hi])
                if c["bias"]:
                    pre[lo:hi] += s["bias"][e].double()
        out = _forward64(c["activation"], pre)
        if c["residual"]:
            out = out + s["residual"].double()
        return {"out": out, "pre": pre} if c["pre"] else {"out": out}
    if op == "input_grad":
        d = torch.empty(off[-1], c["K"], **f64)
        for e in range(c["E"]):
            lo, hi = off[e], off[e + 1]
            if hi > lo:
                torch.mm(s["dy"][lo:hi].double(), s["w"][e].double(), out=d[lo:hi])
        if c["activation"] == "none":
            return {"dx": d}
        v = s["pre"].double()
        if c["activation"] != "swiglu":
            return {"dx": d * _slope64(c["activation"], v)}
        gate, up = v[:, : c["K"]], v[:, c["K"]:]
        return {"dx": torch.cat([d * up * _slope64("silu", gate), d * gate * torch.sigmoid(gate)], 1)}
    dw = torch.zeros(c["E"], c["N"], c["K"], **f64)
    db = torch.zeros(c["E"], c["N"], **f64)
    for e in range(c["E"]):
        lo, hi = off[e], off[e + 1]
        if hi > lo:
            dy = s["dy"][lo:hi].double()
            dw[e] = torch.einsum("rn,rk->nk", dy, s["a"][lo:hi].double())
            db[e] = dy.sum(0)
    return {"dw": dw, "db": db} if c["bias"] else {"dw": dw}
