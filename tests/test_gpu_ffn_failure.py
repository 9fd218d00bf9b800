"""A lost operand load in the product kernels: reported, and nothing left behind.

moe_ffn_test_drop_load makes every CTA leave out one of its loads, as if the
copy never arrived.  Nothing completes the wait for it, the kernel gives up
after its limit (2 s), waits for what it has in flight, reports MOE_ETIMEDOUT
and returns (no trap, no fault, no endless wait).  Then the same call without
the loss is right again."""
import time

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

from test_gpu_decode_layer import ffn, run, tokens, weights  # noqa: E402,F401
from test_gpu_expert_gemm import check_gemm, check_glu, inputs, offsets_of  # noqa: E402


@pytest.fixture()
def drop():
    from combine_route_count_gb300 import moe
    yield moe.moe_ffn_test_drop_load
    moe.moe_ffn_test_drop_load(-1)


def timed_out(call, status):
    from combine_route_count_gb300 import moe
    status.zero_()
    torch.cuda.synchronize()
    t0 = time.monotonic()
    call()
    torch.cuda.synchronize()
    assert int(status) == moe.MOE_ETIMEDOUT
    assert 1.5 < time.monotonic() - t0 < 30.0
    assert torch.cuda.current_stream().query()  # nothing left running


# The rows, experts and K that take the tile kernel, row groups (alone and as a
# cluster) and the few-row kernel (alone and as a cluster).
GEMM = [([300, 100], 512, 1024), ([4] * 16, 640, 40 * 128), ([3, 0, 9], 264, 40 * 128), ([7], 136, 128), ([20], 1024, 6000)]


@pytest.mark.parametrize("counts,N,K", GEMM)
@pytest.mark.parametrize("load", [0, 2])
def test_product_that_loses_a_load(ffn, drop, counts, N, K, load):  # noqa: F811
    if load * 128 >= K:
        pytest.skip("no such load")
    args, off = inputs(1, sum(counts), len(counts), N, K), offsets_of(counts) if len(counts) > 1 else None
    out = torch.empty(sum(counts), N, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    drop(load)
    timed_out(lambda: ffn.expert_gemm_fp8(*args, out, expert_offsets=off, status=status), status)
    ffn.expert_gemm_fp8(*args, out, expert_offsets=off)  # without a status word nothing is reported
    torch.cuda.synchronize()
    drop(-1)
    check_gemm(ffn, *args, off, torch.float32)


@pytest.mark.parametrize("counts", [[300, 100], [2] * 12])
def test_glu_that_loses_a_load(ffn, drop, counts):  # noqa: F811
    args, off = inputs(2, sum(counts), len(counts), 512, 2048), offsets_of(counts)
    q = torch.empty(sum(counts), 256, dtype=torch.uint8, device="cuda")
    s = torch.empty(sum(counts), 2, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    drop(1)
    timed_out(lambda: ffn.expert_glu_fp8(*args, q, s, expert_offsets=off, status=status), status)
    drop(-1)
    check_glu(ffn, *args, off)


@pytest.mark.parametrize("T,H,I,E,K", [(1, 512, 256, 16, 4), (40, 256, 512, 8, 2), (64, 1152, 384, 40, 6)])
def test_layer_that_loses_a_load(ffn, drop, T, H, I, E, K):  # noqa: F811
    ws, tk = weights(3, E, H, I), tokens(4, T, H, K, E)
    layer = ffn.DecodeLayer(T, K, *ws)
    want, out = run(layer, *tk), torch.empty(T, H, dtype=torch.bfloat16, device="cuda")
    drop(1)
    timed_out(lambda: layer.forward(*tk, out), layer.status)
    drop(-1)
    assert torch.equal(run(layer, *tk), want)


def test_values_that_are_refused(ffn):  # noqa: F811
    from combine_route_count_gb300 import moe
    with pytest.raises(moe.MoEError):
        moe.moe_ffn_test_drop_load(-2)
