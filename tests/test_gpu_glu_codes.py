"""moe_expert_glu_fp8's codes one by one against the formula in 64 bits.

Every element has the bound of its own: err for h as ffn_ref.glu derives it,
and for the scale the block's largest err over its largest value.  Rounding is
monotone, so a code lies between those of h - err and h + err.  The inputs are
scaled so that gates are of order 1 and err is far below a code's step:
 - integer codes and scales that are powers of two: gate and up are exact in
   float32, and err is SiLU's and the products' alone, 8 * 2^-23 of h (expf 1
   ulp, the sum 1 + exp, the quotient 2 ulp, three roundings);
 - random codes and scales: also product_error times the sum of magnitudes.
Below about -87.3, where 1 + exp(-gate) passes 2^126, h may be 0: its size is then
below 2^-119 of up."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

import ffn_ref as ref  # noqa: E402
from test_gpu_expert_gemm import blocks, codes, ffn, glu, offsets_of  # noqa: E402,F401

SIZES = [("few", [5] * 16, 256, 256), ("few, long K", [2] * 12, 128, 4096), ("ragged", [0, 1, 130, 0, 7, 128, 64, 257, 3], 640, 1024),
         ("short K", [40, 90], 384, 400), ("dense", [33], 256, 512), ("dense, many", [300], 384, 640)]


def inputs(seed, rows, E, I, H, exact, gate_bits):
    """a, w13 and scales; gates have a standard deviation near 2^gate_bits, ups near 1."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    a, w = codes(g, rows, H, integers=exact), codes(g, E, 2 * I, H, integers=exact)
    sa, sw = torch.ones(rows, blocks(H), device="cuda"), torch.ones(E, 2 * I // 128, blocks(H), device="cuda")
    # A product of codes has the deviation 20/3 (integers of -4 .. 4) or 100 * 100, saturated a little.
    one = 2.0 ** round(-np.log2((20 / 3 if exact else 1e4) * H ** 0.5))
    sw *= one
    sw[:, :I // 128] *= 2.0 ** gate_bits
    if exact:
        sa *= torch.exp2(torch.randint(-1, 2, (rows, 1), generator=g, device="cuda").float())
        sw *= torch.exp2(torch.randint(-1, 2, sw.shape, generator=g, device="cuda").float())
    else:
        sa *= 0.5 + torch.rand(sa.shape, generator=g, device="cuda")
        sw *= 0.5 + torch.rand(sw.shape, generator=g, device="cuda")
    return a, sa, w, sw


def check(ffn, args, off, exact):  # noqa: F811
    q, s = glu(ffn, *args, off)
    q, s = ref.f64(q.view(torch.float8_e4m3fn).float()), ref.f64(s)
    P, S = ref.product(*args, None if off is None else off.tolist())
    I = P.shape[1] // 2
    h, err = ref.glu(P, S, 0.0 if exact else ref.product_error(args[1].shape[1]))
    err = torch.where(P[:, :I] < -87.0, torch.maximum(err, h.abs()), err)
    h, err = ref.f64(h), ref.f64(err)
    want, scale = ref.quantise(h)
    rel = err.reshape(len(h), -1, 128).max(-1) / (scale * 448.0) + 2.0 ** -22
    assert np.all(np.abs(s - scale) <= rel * scale)
    wide, wide_rel = np.repeat(scale, 128, 1), np.repeat(rel, 128, 1)
    slack = np.abs(h) / wide * wide_rel
    lo, hi = ref.e4m3((h - err) / wide - slack), ref.e4m3((h + err) / wide + slack)
    assert np.all((q >= lo) & (q <= hi)), f"{np.mean((q < lo) | (q > hi)):.2e} of the codes"
    # What the bounds leave open is little: few codes may fall to either side, by one step.
    moved = np.abs(q * np.repeat(s, 128, 1) - want * wide)
    assert np.linalg.norm(moved) < (0.002 if exact else 0.02) * np.linalg.norm(want * wide)
    if exact:
        assert np.mean(lo != hi) < 1e-3


@pytest.mark.parametrize("name,counts,I,H", SIZES)
@pytest.mark.parametrize("gate_bits", [0, 2, 5])
def test_exact_products(ffn, name, counts, I, H, gate_bits):  # noqa: F811
    """gate_bits 2: gates to about -15 on the steep side; 5: to far below -87."""
    args = inputs(I + H, sum(counts), len(counts), I, H, True, gate_bits)
    check(ffn, args, None if len(counts) == 1 else offsets_of(counts), True)


@pytest.mark.parametrize("name,counts,I,H", SIZES + [("few, longest K", [3] * 8, 128, 7168)])
def test_random_products(ffn, name, counts, I, H):  # noqa: F811
    args = inputs(I * H, sum(counts), len(counts), I, H, False, 0)
    check(ffn, args, None if len(counts) == 1 else offsets_of(counts), False)


@pytest.mark.parametrize("rows", [8, 300])
def test_blocks_of_small_h(ffn, rows):  # noqa: F811
    """Every gate of a block far on the negative side, with large ups: the scale follows h down to its floor."""
    K, gates = 128, [0.25, 0.5, 1.0, 1.5, 2.0, 2.5, 3.0, 3.5, 4.0, 4.5, 5.0, 5.5]
    I = 128 * len(gates)
    a = torch.zeros(rows, K, device="cuda")
    a[:, 0] = torch.arange(rows, device="cuda") % 8 + 8.0  # 8 .. 15, exact codes
    a[:, 1] = 1.0
    w = torch.zeros(1, 2 * I, K, device="cuda")
    gate = -torch.tensor(gates, device="cuda").repeat_interleave(128)  # times 8 .. 15: -2 to -82.5
    w[0, :I, 0] = gate
    w[0, I:, 1] = 8.0 + torch.arange(I, device="cuda") % 8
    w[0, I::3, 1] *= -1
    sw = torch.ones(1, 2 * I // 128, 1, device="cuda")
    sw[:, I // 128:] = 2.0 ** 10
    args = (a.to(torch.float8_e4m3fn), torch.ones(rows, 1, device="cuda"), w.to(torch.float8_e4m3fn), sw)
    assert torch.equal(args[0].float(), a) and torch.equal(args[2].float(), w)
    check(ffn, args, None, True)
