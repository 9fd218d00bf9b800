"""A lost operand load in the bf16 products' kernels: reported, and nothing left behind.

As for the feed-forward operators: moe_ffn_test_drop_load makes every CTA leave out
one of its loads, the waits for it run out after their limit (2 s), the kernel
reports MOE_ETIMEDOUT and returns.  Then the same call without the loss is right."""
import time

import numpy as np
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def train():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from combine_route_count_gb300 import build, moe, train as t
    build.build()
    build.build_train()
    moe.load_library()
    return t


@pytest.fixture()
def drop():
    from combine_route_count_gb300 import moe
    yield moe.moe_ffn_test_drop_load
    moe.moe_ffn_test_drop_load(-1)


# Rows of each expert, N, K that take one CTA a tile, pairs, a split sum and few rows (one
# CTA, and a cluster): of the forward product.
WAYS = [([100, 60, 0, 90], 512, 512), ([300, 600], 256, 512), ([200], 256, 4096), ([2] * 300, 64, 512), ([3], 264, 2048)]


@pytest.mark.parametrize("counts,N,K", WAYS)
@pytest.mark.parametrize("load", [0, 2])
def test_product_that_loses_a_load(train, drop, counts, N, K, load):
    from combine_route_count_gb300 import moe
    g = torch.Generator(device="cuda").manual_seed(3)
    rows, E = sum(counts), len(counts)
    bf = lambda *s: torch.randint(-2, 3, s, generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
    off = None if E == 1 else torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32, device="cuda")
    a, w, dy = bf(rows, K), bf(E, N, K), bf(rows, N)
    out, dx = torch.empty(rows, N, device="cuda"), torch.empty(rows, K, dtype=torch.bfloat16, device="cuda")
    dw, status = torch.empty(E, N, K, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    calls = {"forward": lambda: train.expert_linear(a, w, out, expert_offsets=off, status=status),
             "by rows": lambda: train.expert_linear_backward_input(dy, w, dx, expert_offsets=off, status=status),
             "by weights": lambda: train.expert_linear_backward_weight(dy, a, dw, expert_offsets=off, status=status)}
    # How many stages the longest sum has, at least, in the CTA that has the fewest of them.
    stages = {"forward": K // 64 // 8, "by rows": N // 64 // 8, "by weights": max(counts) // 64}
    for name, call in calls.items():
        if load >= max(1, stages[name]):
            continue
        call()
        want = (out if name == "forward" else dx if name == "by rows" else dw).clone()
        assert int(status) == moe.MOE_OK
        drop(load)
        t0 = time.monotonic()
        call()
        torch.cuda.synchronize()
        assert int(status) == moe.MOE_ETIMEDOUT, name
        assert 1.5 < time.monotonic() - t0 < 30.0
        assert torch.cuda.current_stream().query()  # nothing left running
        drop(-1)
        status.zero_()
        call()
        assert int(status) == moe.MOE_OK
        assert torch.equal(want, out if name == "forward" else dx if name == "by rows" else dw), name
