"""Cases that time the feed-forward operators around dispatch and combine.

Four operators, all with the block-scaled E4M3 payload of the fp8 dispatch (one float32 scale for each block of 128
elements of a row; weights one scale for each 128 x 128 block):

  norm   residual addition, root-mean-square norm and quantisation of the rows that go into the dispatch
  gemm   the experts' product on grouped rows (or one dense product): bf16 or float32 rows out
  glu    the experts' gate and up product with SiLU(gate) * up, quantised again: the input of the second product
  layer  a whole expert layer for a few tokens: glu, second product and the weighted sum over the chosen experts

``run`` computes them in elementary torch operations in 32 bits, or, with ``own`` set, calls the package.
"""
import math

import torch

own = False

BLOCK = 128
FP8_MAX = 448.0
TINY = 2.0 ** -100  # a block's largest value counts as at least this when its scale is taken


# ---- the cases -----------------------------------------------------------------

def listed():
    return [
        # one sequence's new token in front of an expert layer: latency
        {"name": "norm_token", "op": "norm", "T": 1, "H": 7168, "residual": True, "y": True, "weight": "bf16"},
        # a mixed batch of odd size, first norm of a model (no residual yet), nothing but the 8-bit rows wanted
        {"name": "norm_mixed", "op": "norm", "T": 777, "H": 4224, "residual": False, "y": False, "weight": "f32"},
        # prefill: 64 ranks of 256 tokens
        {"name": "norm_prefill", "op": "norm", "T": 16384, "H": 7168, "residual": True, "y": True, "weight": "bf16"},
        # a shared expert's second product for seven sequences in decode
        {"name": "gemm_few", "op": "gemm", "T": 7, "topk": 1, "E": 1, "N": 7168, "K": 2048, "skew": 0.0, "out": "bf16"},
        # ragged groups under a skewed router, odd sizes in all three directions, float32 rows
        {"name": "gemm_ragged", "op": "gemm", "T": 1001, "topk": 3, "E": 40, "N": 1416, "K": 2320, "skew": 1.0,
         "out": "f32"},
        # the second product of 256 experts over 32 ranks of 128 tokens
        {"name": "gemm_experts", "op": "gemm", "T": 4096, "topk": 8, "E": 256, "N": 7168, "K": 2048, "skew": 0.0,
         "out": "bf16"},
        # one dense projection of a long prefill
        {"name": "gemm_dense", "op": "gemm", "T": 8192, "topk": 1, "E": 1, "N": 7168, "K": 4096, "skew": 0.0,
         "out": "bf16"},
        # 64 tokens over 256 experts: two rows an expert, all the weights are read
        {"name": "glu_decode", "op": "glu", "T": 64, "topk": 8, "E": 256, "H": 7168, "I": 1024, "skew": 0.0},
        # eight experts, a thousand rows each: the tensor cores' case
        {"name": "glu_prefill", "op": "glu", "T": 4096, "topk": 2, "E": 8, "H": 4096, "I": 8192, "skew": 0.0},
        # the smallest layer: 64 tokens, eight small experts: latency
        {"name": "layer_tiny", "op": "layer", "T": 64, "topk": 2, "E": 8, "H": 256, "I": 512, "skew": 0.0},
        # one sequence's new token through eight of 256 experts
        {"name": "layer_token", "op": "layer", "T": 1, "topk": 8, "E": 256, "H": 7168, "I": 2048, "skew": 0.0},
        # an odd batch of decoding sequences under a skewed router
        {"name": "layer_batch", "op": "layer", "T": 37, "topk": 6, "E": 64, "H": 4096, "I": 1408, "skew": 0.5},
    ]


def _spread(rng, lo, hi, step=1):
    """A size between lo and hi, spread over its logarithm, a multiple of step (never 24 * 128)."""
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi))) / step)) * step
    v = min(max(v, step, lo), hi // step * step)
    return v + step if v == 24 * BLOCK else v


def draw(rng):
    op = rng.choice(["norm", "gemm", "glu", "layer"])
    while True:
        if op == "norm":
            residual = rng.random() < 0.7
            c = {"op": op, "T": _spread(rng, 1, 16384), "H": _spread(rng, 128, 16384, 128), "residual": residual,
                 "y": rng.random() < 0.5, "weight": rng.choice(["bf16", "f32"])}
            if c["T"] * c["H"] <= 16384 * 7168:
                return c
            continue
        grouped = op != "gemm" or rng.random() < 0.6
        E = _spread(rng, 2, 384) if grouped else 1
        c = {"op": op, "T": _spread(rng, 1, 37 if op == "layer" else 8192), "topk": min(E, rng.randint(1, 8)), "E": E,
             "skew": rng.choice([0.0, 0.5, 1.0]) if grouped else 0.0}
        if op == "gemm":
            c.update(N=_spread(rng, 128, 8192, 8), K=_spread(rng, 128, 8192, 16), out=rng.choice(["bf16", "f32"]))
            weights = E * c["N"] * c["K"]
        else:
            c.update(H=_spread(rng, 256, 7168, 128), I=_spread(rng, 128, 8192, 128))
            if c["I"] == 12 * BLOCK:
                c["I"] += BLOCK
            weights = E * c["I"] * c["H"] * (2 if op == "glu" else 3)
        if c["T"] * c["topk"] == 24 * BLOCK:
            c["T"] += 1
        if weights <= 3.6e9 and work(c)["flops"] <= 8e11:
            return c


def _experts_with_rows(T, topk, E):
    """How many of E experts T tokens reach, on average, with topk different ones each."""
    return E * (1.0 - (1.0 - topk / E) ** T)


def work(case):
    c = case
    if c["op"] == "norm":
        n = c["T"] * c["H"]
        per = 2 + (4 if c["residual"] else 0) + (2 if c["y"] else 0) + 1
        return {"bytes": n * per + n // BLOCK * 4 + c["H"] * (2 if c["weight"] == "bf16" else 4), "flops": 8 * n}
    T, rows = c["T"], c["T"] * c["topk"]
    active = _experts_with_rows(T, c["topk"], c["E"])
    if c["op"] == "gemm":
        N, K = c["N"], c["K"]
        kb, nb = -(-K // BLOCK), -(-N // BLOCK)
        return {"bytes": rows * (K + 4 * kb) + active * (N * K + 4 * nb * kb) + rows * N * (2 if c["out"] == "bf16" else 4),
                "flops": 2 * rows * N * K}
    H, I = c["H"], c["I"]
    if c["op"] == "glu":
        return {"bytes": rows * (H + H // 32) + active * 2 * I * (H + H // BLOCK / 32) + rows * (I + I // 32),
                "flops": 4 * rows * I * H}
    return {"bytes": T * (H + H // 32) + active * 3 * I * (H + H // BLOCK / 32) + rows * 8 + T * H * 2,
            "flops": 6 * rows * I * H}


# ---- the inputs -----------------------------------------------------------------

def _quantise(v):
    """float32 [rows, n], n a multiple of the block -> E4M3 codes [rows, n], float32 scales [rows, n / 128]."""
    b = v.view(v.shape[0], -1, BLOCK)
    amax = b.abs().amax(-1)
    scale = torch.where(amax > 0, amax.clamp_min(TINY) / FP8_MAX, torch.ones_like(amax))
    q = (b * (1.0 / scale)[..., None]).clamp_(-FP8_MAX, FP8_MAX).to(torch.float8_e4m3fn)
    return q.view(v.shape), scale


def _rows(g, rows, n):
    """Quantised activations: normal values, a few channels much larger, rows of different size."""
    n_up = -(-n // BLOCK) * BLOCK
    v = torch.randn(rows, n_up, generator=g, device="cuda")
    v *= torch.exp(0.5 * torch.randn(rows, 1, generator=g, device="cuda"))
    v[:, :: max(1, n // 4)] *= 8.0
    q, s = _quantise(v)
    return (q if n_up == n else q[:, :n].contiguous()), s


def _weights(g, E, n, k):
    """Quantised weights [E, n, k] as a checkpoint holds them, one scale for each 128 x 128 block."""
    w = torch.randn(E, n, k, generator=g, device="cuda", dtype=torch.bfloat16)
    w = w.mul_(107.0).clamp_(-FP8_MAX, FP8_MAX).to(torch.float8_e4m3fn)
    s = torch.rand(E, -(-n // BLOCK), -(-k // BLOCK), generator=g, device="cuda")
    return w, (0.5 + s) * (1.0 / (107.0 * math.sqrt(k)))


def _choices(g, T, topk, E, skew):
    """topk different experts for each token and their weights, popularity spread by skew."""
    popularity = skew * torch.randn(1, E, generator=g, device="cuda")
    u = torch.rand(T, E, generator=g, device="cuda").clamp_(1e-7, 1.0 - 1e-7)
    score, idx = torch.topk(popularity - torch.log(-torch.log(u)), topk, dim=1)
    return idx.to(torch.int32), torch.softmax(score, 1)


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    s = {"case": c}
    empty = dict(device="cuda")
    if c["op"] == "norm":
        T, H = c["T"], c["H"]
        x = torch.randn(T, H, generator=g, device="cuda")
        x[:, :: H // 4] *= 20.0
        s["x"] = x.to(torch.bfloat16)
        s["residual"] = (3.0 * torch.randn(T, H, generator=g, device="cuda")).to(torch.bfloat16) if c["residual"] else None
        w = 1.0 + 0.2 * torch.randn(H, generator=g, device="cuda")
        s["weight"] = w.to(torch.bfloat16) if c["weight"] == "bf16" else w
        s["residual_out"] = torch.empty(T, H, dtype=torch.bfloat16, **empty) if c["residual"] else None
        s["y"] = torch.empty(T, H, dtype=torch.bfloat16, **empty) if c["y"] else None
        s["xq"] = torch.empty(T, H, dtype=torch.float8_e4m3fn, **empty)
        s["scales"] = torch.empty(T, H // BLOCK, dtype=torch.float32, **empty)
        return s
    T, topk, E = c["T"], c["topk"], c["E"]
    rows = T * topk
    if c["op"] == "layer":
        H, I = c["H"], c["I"]
        s["idx"], s["weights"] = _choices(g, T, topk, E, c["skew"])
        s["a"], s["a_scales"] = _rows(g, T, H)
        s["w13"], s["w13_scales"] = _weights(g, E, 2 * I, H)
        s["w2"], s["w2_scales"] = _weights(g, E, H, I)
        s["out"] = torch.empty(T, H, dtype=torch.bfloat16, **empty)
        if own:  # the handle that a program keeps for one layer's weights
            from combine_route_count_gb300 import ffn
            s["layer"] = ffn.DecodeLayer(T, topk, s["w13"], s["w13_scales"], s["w2"], s["w2_scales"])
        return s
    s["offsets"], s["most"] = None, rows
    if E > 1:  # what a dispatch of these tokens leaves in its layout
        idx, _ = _choices(g, T, topk, E, c["skew"])
        counts = torch.bincount(idx.flatten().long(), minlength=E)
        s["offsets"] = torch.cat([torch.zeros_like(counts[:1]), counts.cumsum(0)]).to(torch.int32)
        s["most"] = int(counts.max())
    if c["op"] == "gemm":
        s["a"], s["a_scales"] = _rows(g, rows, c["K"])
        s["w"], s["w_scales"] = _weights(g, E, c["N"], c["K"])
        s["out"] = torch.empty(rows, c["N"], dtype=torch.bfloat16 if c["out"] == "bf16" else torch.float32, **empty)
    else:
        s["a"], s["a_scales"] = _rows(g, rows, c["H"])
        s["w"], s["w_scales"] = _weights(g, E, 2 * c["I"], c["H"])
        s["hq"] = torch.empty(rows, c["I"], dtype=torch.float8_e4m3fn, **empty)
        s["h_scales"] = torch.empty(rows, c["I"] // BLOCK, dtype=torch.float32, **empty)
    return s


# ---- one pass -------------------------------------------------------------------

def _rows_f32(q, scales):
    return q.float().mul_(scales.repeat_interleave(BLOCK, 1)[:, : q.shape[1]])


def _weights_f32(q, scales):
    n, k = q.shape[1:]
    return q.float().mul_(scales.repeat_interleave(BLOCK, 1)[:, :n].repeat_interleave(BLOCK, 2)[:, :, :k])


def _product(s):
    """Grouped rows times their expert's weights, float32 [rows, n]: the groups side by side, padded to the largest."""
    a, w = _rows_f32(s["a"], s["a_scales"]), _weights_f32(s["w"], s["w_scales"])
    if s["offsets"] is None:
        return a @ w[0].t()
    off, most, E = s["offsets"].long(), s["most"], w.shape[0]
    row = torch.arange(a.shape[0], device=a.device)
    e = torch.searchsorted(off[1:], row, right=True)
    at = e * most + row - off[e]
    padded = a.new_zeros(E * most, a.shape[1])
    padded[at] = a
    return torch.bmm(padded.view(E, most, -1), w.transpose(1, 2)).view(E * most, -1)[at]


def _glu(gu):
    gate, up = gu.chunk(2, -1)
    return gate / (1.0 + torch.exp(-gate)) * up


def _plain(s):
    c = s["case"]
    if c["op"] == "norm":
        v = s["x"].float()
        if c["residual"]:
            v = v + s["residual"].float()
        y = v * torch.rsqrt(v.square().mean(-1, keepdim=True) + 1e-6) * s["weight"].float()
        q, scales = _quantise(y)
        out = {"xq": q, "scales": scales}
        if c["residual"]:
            out["residual"] = v.to(torch.bfloat16)
        if c["y"]:
            out["y"] = y.to(torch.bfloat16)
        return out
    if c["op"] == "gemm":
        return {"out": _product(s).to(s["out"].dtype)}
    if c["op"] == "glu":
        q, scales = _quantise(_glu(_product(s)))
        return {"hq": q, "scales": scales}
    idx, x = s["idx"].long(), _rows_f32(s["a"], s["a_scales"])
    T, topk = idx.shape
    E, I = c["E"], c["I"]
    token = torch.arange(T, device=x.device)[:, None]
    if T * topk < E:  # fewer choices than experts: gather the chosen ones' weights
        flat = idx.flatten()
        w13 = _weights_f32(s["w13"].view(torch.uint8)[flat].view(torch.float8_e4m3fn), s["w13_scales"][flat])
        w2 = _weights_f32(s["w2"].view(torch.uint8)[flat].view(torch.float8_e4m3fn), s["w2_scales"][flat])
        gu = torch.bmm(w13, x.repeat_interleave(topk, 0)[..., None])[..., 0]
        h = _rows_f32(*_quantise(_glu(gu)))
        y = torch.bmm(w2, h[..., None])[..., 0].view(T, topk, -1)
    else:  # else every expert on every token
        gu = torch.matmul(x, _weights_f32(s["w13"], s["w13_scales"]).transpose(1, 2))[idx, token].view(T * topk, -1)
        h = x.new_zeros(E, T, I)
        h[idx, token] = _rows_f32(*_quantise(_glu(gu))).view(T, topk, I)
        y = torch.bmm(h, _weights_f32(s["w2"], s["w2_scales"]).transpose(1, 2))[idx, token]
    return {"out": (s["weights"][..., None] * y).sum(1).to(torch.bfloat16)}


def _own(s):
    from combine_route_count_gb300 import ffn
    c = s["case"]
    if c["op"] == "norm":
        ffn.add_rms_norm_fp8(s["x"], s["weight"], s["xq"], s["scales"], eps=1e-6, residual=s["residual"],
                             residual_out=s["residual_out"], y=s["y"])
        out = {"xq": s["xq"], "scales": s["scales"]}
        if c["residual"]:
            out["residual"] = s["residual_out"]
        if c["y"]:
            out["y"] = s["y"]
        return out
    if c["op"] == "gemm":
        ffn.expert_gemm_fp8(s["a"], s["a_scales"], s["w"], s["w_scales"], s["out"], expert_offsets=s["offsets"])
        return {"out": s["out"]}
    if c["op"] == "glu":
        ffn.expert_glu_fp8(s["a"], s["a_scales"], s["w"], s["w_scales"], s["hq"], s["h_scales"],
                           expert_offsets=s["offsets"])
        return {"hq": s["hq"], "scales": s["h_scales"]}
    s["layer"].forward(s["a"], s["a_scales"], s["idx"], s["weights"], s["out"])
    return {"out": s["out"]}


def run(state):
    return _own(state) if own else _plain(state)


# ---- the definition in 64 bits ---------------------------------------------------

def _e4m3(v):
    """The nearest E4M3 values (ties to even, saturating) of float64 values."""
    _, e = torch.frexp(v.abs().clamp_min(2.0 ** -6))  # |v| < 2^e; three bits after the leading one
    step = torch.exp2(e.double() - 4.0)
    return (torch.round(v / step) * step).clamp_(-FP8_MAX, FP8_MAX)


def _codes64(v):
    """float64 rows -> (values of the codes, scales), block by block."""
    b = v.reshape(v.shape[0], -1, BLOCK)
    top = b.abs().amax(2, keepdim=True)
    scale = torch.where(top > 0, torch.maximum(top, torch.full_like(top, TINY)) / FP8_MAX, torch.ones_like(top))
    return _e4m3(b / scale).reshape(v.shape), scale[..., 0]


def _a64(q, scales):
    """Quantised rows as float64 values."""
    column = torch.arange(q.shape[1], device=q.device) // BLOCK
    return q.double() * scales.double()[:, column]


def _w64(q, scales):
    """One expert's quantised weights as float64 values."""
    r = torch.arange(q.shape[0], device=q.device) // BLOCK
    k = torch.arange(q.shape[1], device=q.device) // BLOCK
    return q.double() * scales.double()[r][:, k]


def _silu64(gu):
    n = gu.shape[1] // 2
    return gu[:, :n] * torch.sigmoid(gu[:, :n]) * gu[:, n:]


def exact(case, seed):
    if work(case)["flops"] > 4e12:
        return None
    s, c = prepare(case, seed), case
    if c["op"] == "norm":
        v = s["x"].double()
        if c["residual"]:
            v += s["residual"].double()
        y = v / torch.sqrt((v * v).sum(1, keepdim=True) / c["H"] + 1e-6) * s["weight"].double()
        q, scale = _codes64(y)
        out = {"xq": q, "scales": scale}
        if c["residual"]:
            out["residual"] = v
        if c["y"]:
            out["y"] = y
        return out
    if c["op"] == "layer":
        out = torch.zeros(c["T"], c["H"], dtype=torch.float64, device="cuda")
        x, idx = _a64(s["a"], s["a_scales"]), s["idx"]
        for e in sorted(set(idx.flatten().tolist())):
            t, k = (idx == e).nonzero(as_tuple=True)
            h = _silu64(x[t] @ _w64(s["w13"][e], s["w13_scales"][e]).t())
            q, scale = _codes64(h)
            y = (q * scale.repeat_interleave(BLOCK, 1)) @ _w64(s["w2"][e], s["w2_scales"][e]).t()
            out[t] += s["weights"].double()[t, k][:, None] * y
        return {"out": out}
    off = [0, s["a"].shape[0]] if s["offsets"] is None else s["offsets"].tolist()
    n = s["w"].shape[1]
    p = torch.empty(s["a"].shape[0], n, dtype=torch.float64, device="cuda")
    for e, (lo, hi) in enumerate(zip(off[:-1], off[1:])):
        if hi > lo:
            p[lo:hi] = _a64(s["a"][lo:hi], s["a_scales"][lo:hi]) @ _w64(s["w"][e], s["w_scales"][e]).t()
    if c["op"] == "gemm":
        return {"out": p}
    q, scale = _codes64(_silu64(p))
    return {"hq": q, "scales": scale}
