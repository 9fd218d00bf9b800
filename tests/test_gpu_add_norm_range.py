"""moe_add_rms_norm_fp8 where s * weight is small and 1 / sqrt(mean(s^2) + eps) large.

What include/moe_ffn.h promises holds wherever the squares of s and s * weight
are normal float32 numbers, however small eps and the weights are.  Tolerances
are those of test_gpu_add_norm.py: every v within REL of its own size."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

import ffn_ref as ref  # noqa: E402
from test_gpu_add_norm import REL, check, ffn, run  # noqa: E402,F401


def small(rng, T, H, exponent):
    """bf16 values of either sign, sizes within a factor of four of 2^exponent, an eighth of them zero."""
    v = rng.choice([-1.0, 1.0], (T, H)) * 2.0 ** rng.uniform(-1, 1, (T, H)) * (rng.random((T, H)) > 0.125)
    return torch.from_numpy((v * 2.0 ** exponent).astype(np.float32)).to(torch.bfloat16)


# (eps, log2 of s, log2 of the weight): s * weight from 2^-120 on, above and below the scales' floor of 2^-100 after the norm
SMALL = [(1e-30, -50, -70), (1e-38, -60, -60), (1e-38, -60, -40), (1e-12, -60, -59), (1e-12, -60, -30), (1e-6, -60, -59),
         (1e-45, -58, -50), (1e-45, 0, -118), (1e-20, -20, -99)]


@pytest.mark.parametrize("eps,xe,we", SMALL)
@pytest.mark.parametrize("H", [512, 16512])
@pytest.mark.parametrize("residual", [True, False])
def test_small_values_and_weights(ffn, eps, xe, we, H, residual):  # noqa: F811
    rng = np.random.default_rng(H - xe - we)
    x, w = small(rng, 5, H, xe), small(rng, 1, H, we)[0].float()
    x[1] = 0
    x[2, 128:256] = 0
    eps = float(np.float32(eps))
    check(ffn, x, w, small(rng, 5, H, xe - 3) if residual else None, eps=eps)


def test_blocks_of_every_size_in_one_row(ffn):  # noqa: F811
    """A warp that holds blocks far below the floor and blocks far above it: each keeps its own arithmetic."""
    rng = np.random.default_rng(3)
    H = 128 * 40
    x = small(rng, 3, H, -55)
    w = torch.from_numpy(np.repeat(2.0 ** (-1.6 * np.arange(40)), 128).astype(np.float32))
    w[rng.permutation(H)[:100]] = 0
    eps = float(np.float32(1e-36))
    check(ffn, x, w, eps=eps)
    # Blocks that are not small have the codes and scales that they have among others of their size.
    q, s, _, _ = run(ffn, x, w, eps=eps)
    alone = w.clone()
    alone[128 * 8:] = 1.0
    q1, s1, _, _ = run(ffn, x, alone, eps=eps)
    assert np.array_equal(q[:, :128 * 8], q1[:, :128 * 8]) and np.array_equal(s[:, :8], s1[:, :8])
