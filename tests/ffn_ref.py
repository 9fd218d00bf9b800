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
    kernel's v may be off by a relative `rel` of its block's largest value:
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
    assert np.all(far <= 0.5 * step + 3 * rel * 448.0), np.max(far - 0.5 * step)


def add_norm(x, residual, weight, eps):
    s = x + residual if residual is not None else x
    return s, s / np.sqrt((s * s).mean(-1, keepdims=True) + eps) * weight
