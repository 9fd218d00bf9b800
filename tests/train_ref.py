"""Plain implementations in 64 bits of the training operators, for tests.

Written from the formulas of include/moe_train.h on torch float64; nothing here
calls the package.  What rounds is counted in steps of the type's spacing:
half a step is eps / 2 of the value (bf16 2^-9 of its binade's top, i.e. at most
2^-8 of the value; float32 2^-24)."""
import math

import torch

F32 = 2.0 ** -24


def half_step(v, dtype):
    """Most that rounding v to dtype moves it (plus a subnormal's half step)."""
    if dtype == torch.float32:
        return v.abs() * F32 + 2.0 ** -150
    return v.abs() * 2.0 ** -8 + 2.0 ** -134


def near(got, want, error, dtype=None):
    """got (rounded once to its type) against 64-bit want, off by at most `error` before that rounding."""
    dtype = dtype or got.dtype
    bound = error + half_step(want.abs() + error, dtype)
    far = (got.double() - want).abs()
    assert bool((far <= bound).all()), (float((far / bound.clamp_min(1e-300)).max()), float(far.max()))


# ---- router ---------------------------------------------------------------------

def scores(z, score):
    return torch.sigmoid(z) if score == "sigmoid" else torch.softmax(z, 1)


def choice(z, bias, topk):
    """The topk largest keys, the largest first, the lower index first among equals."""
    key = z if bias is None else torch.sigmoid(z) + bias
    return torch.sort(key, dim=1, descending=True, stable=True)[1][:, :topk]


def weights(z, idx, score, normalize, scale):
    log_p = torch.nn.functional.logsigmoid(z) if score == "sigmoid" else torch.log_softmax(z, 1)
    chosen = log_p.gather(1, idx)
    return scale * (torch.softmax(chosen, 1) if normalize else chosen.exp())


# ---- products ---------------------------------------------------------------------

def clamped(offsets, rows, E):
    if offsets is None:
        return [(0, rows)]
    off = [min(max(int(o), 0), rows) for o in offsets]
    return [(off[e], max(off[e], off[e + 1])) for e in range(E)]


def forward(a, w, offsets):
    """(v, sum of magnitudes), zeros in rows that no expert owns."""
    v = torch.zeros(a.shape[0], w.shape[1], dtype=torch.float64, device=a.device)
    s = torch.zeros_like(v)
    for e, (lo, hi) in enumerate(clamped(offsets, a.shape[0], w.shape[0])):
        x, y = a[lo:hi].double(), w[e].double()
        v[lo:hi], s[lo:hi] = x @ y.t(), x.abs() @ y.abs().t()
    return v, s


def by_rows(dy, w, offsets):
    g = torch.zeros(dy.shape[0], w.shape[2], dtype=torch.float64, device=dy.device)
    s = torch.zeros_like(g)
    for e, (lo, hi) in enumerate(clamped(offsets, dy.shape[0], w.shape[0])):
        x, y = dy[lo:hi].double(), w[e].double()
        g[lo:hi], s[lo:hi] = x @ y, x.abs() @ y.abs()
    return g, s


def by_weights(dy, a, offsets, E):
    dw = torch.zeros(E, dy.shape[1], a.shape[1], dtype=torch.float64, device=a.device)
    s = torch.zeros_like(dw)
    db = torch.zeros(E, dy.shape[1], dtype=torch.float64, device=a.device)
    sb = torch.zeros_like(db)
    for e, (lo, hi) in enumerate(clamped(offsets, a.shape[0], E)):
        x, y = dy[lo:hi].double(), a[lo:hi].double()
        dw[e], s[e] = x.t() @ y, x.abs().t() @ y.abs()
        db[e], sb[e] = x.sum(0), x.abs().sum(0)
    return dw, s, db, sb


def product_error(kc):
    """Of a sum of kc exact products over its sum of magnitudes: every addition may truncate (2^-23)."""
    return (kc + 1) * 2.0 ** -23


def act(name, v):
    if name == "relu":
        return v.clamp_min(0)
    if name == "gelu":
        return v * 0.5 * torch.erfc(-v / math.sqrt(2))
    if name == "silu":
        return v * torch.sigmoid(v)
    if name == "swiglu":
        n = v.shape[1] // 2
        return v[:, :n] * torch.sigmoid(v[:, :n]) * v[:, n:]
    return v


def act_error(name, v, err):
    """Bound on the error of act(v) in float32 with v off by err: |act'| <= 1.13
    (gelu's largest slope), erf and exp within 2 ulp, a quotient within 2 ulp (of
    a denominator within 2.5), the factors and sums rounded: 10 steps of |v| in
    all (swiglu: of the product's factors)."""
    if name == "swiglu":
        n = v.shape[1] // 2
        gate, up, eg, eu = v[:, :n], v[:, n:], err[:, :n], err[:, n:]
        silu = gate * torch.sigmoid(gate)
        return 1.13 * eg * (up.abs() + eu) + silu.abs() * eu + 12 * F32 * 2 * silu.abs() * up.abs() + 1e-37
    if name == "none":
        return err
    return 1.13 * err + 20 * F32 * v.abs() + 1e-37


def slope(name, v):
    if name == "relu":
        return (v > 0).double()
    if name == "gelu":
        return 0.5 * torch.erfc(-v / math.sqrt(2)) + v * torch.exp(-v * v / 2) / math.sqrt(2 * math.pi)
    s = torch.sigmoid(v)
    return s * (1 + v * (1 - s))


def through(name, g, err, v):
    """(gradient, error bound) of g (off by err) through the activation at v.  The
    slope in float32: its terms are at most 1 + |v| and a few roundings off."""
    if name == "none":
        return g, err
    if name == "swiglu":
        n = v.shape[1] // 2
        gate, up = v[:, :n], v[:, n:]
        silu = gate * torch.sigmoid(gate)
        d = torch.cat([g * up * slope("silu", gate), g * silu], 1)
        e = torch.cat([err * up.abs() * 1.13 + 24 * F32 * g.abs() * up.abs() * (1 + gate.abs()),
                       err * silu.abs() + 24 * F32 * g.abs() * gate.abs()], 1)
        return d, e + 1e-37
    return g * slope(name, v), 1.13 * err + 24 * F32 * g.abs() * (1 + v.abs()) + 1e-37
