"""Grouped products of a skewed router at a layer's size: few of many experts have all the rows."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

from test_gpu_expert_gemm import check_gemm, check_glu, ffn, inputs, offsets_of  # noqa: E402,F401


@pytest.mark.parametrize("rows", [512, 1024, 2048])
@pytest.mark.parametrize("hot", [1, 8, 40])
def test_rows_on_few_experts(ffn, rows, hot):  # noqa: F811
    E = 256
    rng = np.random.default_rng(rows + hot)
    counts = np.zeros(E, np.int64)
    counts[rng.permutation(E)[:hot]] = rng.multinomial(rows, np.ones(hot) / hot)
    off = offsets_of(counts)
    check_glu(ffn, *inputs(hot, rows, E, 2 * 256, 7168), off)
    check_gemm(ffn, *inputs(hot, rows, E, 264, 7168), off, torch.bfloat16)
