"""More units of a few rows than CTAs, with a long K: the last ones are split along K over a cluster's CTAs.
(Sizes with and without units left over, and with some left that are too many to split.)"""
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

from test_gpu_decode_layer import check as check_layer  # noqa: E402
from test_gpu_expert_gemm import check_gemm, check_glu, ffn, inputs, offsets_of  # noqa: E402,F401


@pytest.mark.parametrize("counts,I", [([2] * 31, 1280), ([2] * 38, 1024), ([3, 0, 1, 17] * 10, 1152), ([2] * 61, 1280)])
@pytest.mark.parametrize("H", [32 * 128, 33 * 128 + 16])
def test_glu(ffn, counts, I, H):  # noqa: F811
    check_glu(ffn, *inputs(I + H, sum(counts), len(counts), 2 * I, H), offsets_of(counts))


@pytest.mark.parametrize("counts,N", [([2] * 31, 2560), ([3, 0, 1, 17] * 10, 2312), ([1] * 64, 2568)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_gemm(ffn, counts, N, dtype):  # noqa: F811
    check_gemm(ffn, *inputs(N, sum(counts), len(counts), N, 33 * 128 + 16), offsets_of(counts), dtype)


@pytest.mark.parametrize("T,H,I,E,K", [(64, 4096, 1280, 31, 2), (64, 4096, 1408, 28, 4), (17, 4096, 1024, 45, 4), (64, 2048, 1280, 31, 2)])
def test_layer(ffn, T, H, I, E, K):  # noqa: F811
    check_layer(ffn, T, H, I, E, K)
