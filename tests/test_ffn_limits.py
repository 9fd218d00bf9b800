"""Sizes next to 2^31 of the product calls: refused on the host where a tile or a block would end past it."""
import pytest

from test_ffn_host import moe, refused  # noqa: F401


@pytest.mark.parametrize("E,n,k", [(1, 256, 2 ** 31 - 16), (1, 256, 2 ** 31 - 112), (1, 2 ** 31 - 8, 16),
                                   (1, 2 ** 31 - 248, 16), (8, 2 ** 28 - 8, 16)])
def test_gemm(moe, E, n, k):  # noqa: F811
    A = 0x1000  # never read
    assert refused(moe, moe.moe_expert_gemm_fp8, A, A, 1, k, A, A, n, E, A if E > 1 else None, A, 0, None)


@pytest.mark.parametrize("E,inter,hidden", [(1, 128, 2 ** 31 - 16), (1, 2 ** 30, 16), (4, 2 ** 28, 16)])
def test_glu(moe, E, inter, hidden):  # noqa: F811
    A = 0x1000
    assert refused(moe, moe.moe_expert_glu_fp8, A, A, 1, hidden, A, A, inter, E, A if E > 1 else None, A, A, None)
