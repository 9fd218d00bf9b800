"""Plain implementations in 64 bits of the feed-forward operators, for tests.

Written from the formulas of include/moe_ffn.h on numpy float64; nothing here
calls the package's kernels.  E4M3 codes are handled as the values they stand
for."""
import numpy as np

BLOCK = 128
TINY = 2.0 ** -100


def bf16(rng, *shape, scale=1.0):
    """Random bf16 values as a torch tensor on the CPU."""
    import torch
    return torch.from_numpy((rng.standard_normal(shape) * scale).astype(np.float32)).to(torch.bfloat16)


def f64(t):
    return t.detach().cpu().double().numpy()


def e4m3(v):
    """Nearest E4M3 values, ties to even, saturating at 448."""
    v = np.asarray(v, np.float64)
    _, e = np.frexp(np.maximum(np.abs(v), 2.0 ** -6))
    step = np.exp2(e - 4.0)
    return np.clip(np.round(v / step) * step, -448.0, 448.0)


def quantise(v):
    """float64 rows [n, m*128] -> (values of the codes, scales), exactly by the rule."""
    b = v.reshape(v.shape[0], -1, BLOCK)
    top = np.abs(b).max(-1) if b.size else np.zeros(b.shape[:2])
    scale = np.where(top > 0, np.maximum(top, TINY) / 448.0, 1.0)
    return e4m3(b / scale[..., None]).reshape(v.shape), scale


def dequantise(q, scales):
    """Rows of code values and their block scales -> float64 values (the last block may be short)."""
    return q * np.repeat(scales, BLOCK, axis=1)[:, : q.shape[1]]


def assert_codes_near(q, scales, v, rel):
    """q (code values) and scales against unquantised float64 rows v, where the
    kernel's v may be off by a relative `rel` of its block's largest value (one
    number, or one for each block):
    scales within rel, and each code within half a step of E4M3 (at its
    binade) plus what `rel` moves it by."""
    b = v.reshape(v.shape[0], -1, BLOCK)
    top = np.abs(b).max(-1)
    want = np.where(top > 0, np.maximum(top, TINY) / 448.0, 1.0)
    assert np.all(np.abs(scales - want) <= rel * want), np.max(np.abs(scales / want - 1))
    u = b / want[..., None]
    _, e = np.frexp(np.maximum(np.abs(u) * (1 + 1e-9), 2.0 ** -6))
    step = np.exp2(e - 4.0)
    # A value just below a binade may round up into it, where steps are twice
    # as wide; half a step of the own binade still bounds the distance.
    far = np.abs(q.reshape(b.shape) - u)
    slack = 3 * np.broadcast_to(rel, want.shape)[..., None] * 448.0
    assert np.all(far <= 0.5 * step + slack), np.max(far - 0.5 * step)


def add_norm(x, residual, weight, eps):
    s = x + residual if residual is not None else x
    return s, s / np.sqrt((s * s).mean(-1, keepdims=True) + eps) * weight


def product(a, a_scales, w, w_scales, offsets=None):
    """Grouped product in float64 on the tensors' device, and the same sum over magnitudes.

    a E4M3 [rows, K], w E4M3 [E, N, K]; returns (P, S) with P = 0 in rows no expert owns."""
    import torch
    rows, E = a.shape[0], w.shape[0]
    off = [0, rows] if offsets is None else [min(max(int(o), 0), rows) for o in offsets]
    P = torch.zeros(rows, w.shape[1], dtype=torch.float64, device=a.device)
    S = torch.zeros_like(P)
    k = torch.arange(a.shape[1], device=a.device) // BLOCK
    n = torch.arange(w.shape[1], device=a.device) // BLOCK
    for e in range(E):
        lo, hi = off[e], max(off[e], off[e + 1])
        if hi > lo:
            x = a[lo:hi].float().double() * a_scales[lo:hi].double()[:, k]
            y = w[e].float().double() * w_scales[e].double()[n][:, k]
            P[lo:hi], S[lo:hi] = x @ y.t(), x.abs() @ y.abs().t()
    return P, S


def product_error(kblocks):
    """Bound on a product's error over its sum of magnitudes: up to 128 additions
    inside a block that may truncate (2^-23 each), one scaling and one
    addition for each block in float32, and the product of the two scales."""
    return (128 + kblocks + 3) * 2.0 ** -23


def glu(P, S, rel):
    """h from a gate/up product and a bound on its error: |silu'| < 1.1, float32 exp, division and products."""
    import torch
    I = P.shape[1] // 2
    gate, up, sg, su = P[:, :I], P[:, I:], S[:, :I] * rel, S[:, I:] * rel
    silu = gate * torch.sigmoid(gate)
    h = silu * up
    return h, 1.1 * sg * (up.abs() + su) + silu.abs() * su + 8 * 2.0 ** -23 * h.abs()


def decode_layer(x, sx, idx, weights, w13, s13, w2, s2):
    """The whole layer in float64 (tensors on one device), and a bound on a float32 kernel's error.

    h is quantised by the rule, so its codes may fall to either side of a
    rounding boundary that h is within its own error of: the bound takes the
    codes of h - err and h + err (rounding is monotone)."""
    import torch
    T, K = idx.shape
    H, I = w2.shape[1:]
    out = torch.zeros(T, H, dtype=torch.float64, device=x.device)
    bound = torch.zeros_like(out)
    for e in sorted(set(idx.flatten().tolist())):
        t, k = (idx == e).nonzero(as_tuple=True)
        rel = product_error(sx.shape[1])
        P, S = product(x[t], sx[t], w13[e:e + 1], s13[e:e + 1])
        h, err = glu(P, S, rel)
        h, err = f64(h), f64(err)
        q, scale = quantise(h)
        shape = (len(h), -1, BLOCK)
        top_err = err.reshape(shape).max(-1)
        wide = np.repeat(scale, BLOCK, 1)
        srel = np.repeat(top_err / (scale * 448.0) + 2.0 ** -22, BLOCK, 1)
        lo = e4m3((h - err) / wide - np.abs(h) / wide * srel)
        hi = e4m3((h + err) / wide + np.abs(h) / wide * srel)
        value = q * wide
        dev = np.maximum(np.abs(hi * wide - value), np.abs(value - lo * wide)) + srel * np.abs(value) * 2
        n = torch.arange(H, device=x.device) // BLOCK
        c = torch.arange(I, device=x.device) // BLOCK
        w = w2[e].float().double() * s2[e].double()[n][:, c]
        value, dev = torch.from_numpy(value).to(x.device), torch.from_numpy(dev).to(x.device)
        r = weights.double()[t, k][:, None]
        out[t] += r * (value @ w.t())
        bound[t] += r.abs() * ((dev + product_error(s2.shape[2]) * value.abs()) @ w.abs().t())
    bound += (K + 8) * 2.0 ** -23 * bound + (K + 8 * K) * 2.0 ** -23 * out.abs()
    _, ex = torch.frexp(out.abs() + bound)
    return out, bound + torch.exp2(ex.double() - 9)
