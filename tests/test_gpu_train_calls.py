"""How the training operators are called: refusals on tensors, threads, streams."""
import threading

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


def bf(*s):
    return torch.zeros(*s, dtype=torch.bfloat16, device="cuda")


def f32(*s):
    return torch.zeros(*s, device="cuda")


def i32(*s):
    return torch.zeros(*s, dtype=torch.int32, device="cuda")


def refused(call, what):
    from combine_route_count_gb300 import moe
    with pytest.raises(moe.MoEError) as e:
        call()
    assert e.value.code == moe.MOE_EINVAL and what in str(e.value), str(e.value)


def test_refusals(train):
    z, i, w = f32(4, 8), i32(4, 2), f32(4, 2)
    for call, what in (
            (lambda: train.router_topk(z.cpu(), i, w), "logits must be on the current CUDA device"),
            (lambda: train.router_topk(z.half(), i, w), "logits must be of type"),
            (lambda: train.router_topk(z, i.long(), w), "topk_idx must be of type"),
            (lambda: train.router_topk(z, i, w[:3]), "topk_w must have the shape"),
            (lambda: train.router_topk(z, i, w, bias=f32(7), score="sigmoid"), "bias must have the shape"),
            (lambda: train.router_topk(z, i, w, bias=f32(8)), "moe_router_topk"),
            (lambda: train.router_topk(z, i, w, score="relu"), "score must be one of"),
            (lambda: train.router_topk(z, i, w, scale=float("nan")), "moe_router_topk"),
            (lambda: train.router_topk(z, i32(4, 9), f32(4, 9)), "moe_router_topk"),
            (lambda: train.router_topk(z.t(), i, w), "contiguous"),
            (lambda: train.router_topk(f32(8, 4).t(), i, w), "contiguous"),
            (lambda: train.router_topk_backward(z, i, w, bf(4, 8)), "the logits' type"),
            (lambda: train.combine_backward(bf(4, 64), i, w, bf(8, 64), expert_y=bf(8, 64)), "go together"),
            (lambda: train.combine_backward(bf(4, 64), i, w, bf(8, 56), expert_y=bf(8, 64), d_topk_w=w), "d_expert_y must"),
            (lambda: train.combine_backward(bf(4, 60), i, w, bf(8, 60)), "moe_combine_backward"),
            (lambda: train.dispatch_backward(bf(8, 64), i, bf(5, 64)), "slot_row must have the shape"),
            (lambda: train.dispatch_backward(bf(8, 64), i, bf(4, 64), add=f32(4, 64)), "add must be of type"),
            (lambda: train.expert_linear(bf(4, 64), bf(2, 32, 64), bf(4, 32)), "moe_expert_linear"),
            (lambda: train.expert_linear(bf(4, 64), bf(32, 72), bf(4, 32)), "w must have the shape"),
            (lambda: train.expert_linear(bf(4, 64), bf(32, 64), bf(4, 32), activation="swiglu"), "out must have the shape"),
            (lambda: train.expert_linear(bf(4, 64), bf(24, 64), bf(4, 12), activation="swiglu"), "moe_expert_linear"),
            (lambda: train.expert_linear(bf(4, 64), bf(32, 64), bf(4, 32), activation="tanh"), "activation must be one of"),
            (lambda: train.expert_linear(bf(4, 64), bf(32, 64), bf(4, 32), bias=f32(1, 32)), "bias must have the shape"),
            (lambda: train.expert_linear(bf(4, 64), bf(2, 32, 64), bf(4, 32), expert_offsets=i32(2)), "expert_offsets must"),
            (lambda: train.expert_linear(bf(4, 66)[:, 2:], bf(32, 64), bf(4, 32)), "a must be contiguous"),
            (lambda: train.expert_linear(bf(260)[4:].view(4, 64), bf(32, 64), bf(4, 32)), "moe_expert_linear"),
            (lambda: train.expert_linear_backward_input(bf(4, 32), bf(32, 64), bf(4, 64), activation="silu"), "go together"),
            (lambda: train.expert_linear_backward_input(bf(4, 32), bf(32, 64), bf(4, 64), pre=bf(4, 64)), "go together"),
            (lambda: train.expert_linear_backward_weight(bf(4, 32), bf(4, 64), bf(32, 64), db=bf(32)), "db must be of type"),
            (lambda: train.expert_linear_backward_weight(bf(4, 32), bf(5, 64), bf(32, 64)), "a must have the shape")):
        refused(call, what)
    torch.cuda.synchronize()


def test_threads_whose_first_cuda_call_is_a_product(train):
    """Several threads at once, each on a stream of its own."""
    g = torch.Generator(device="cuda").manual_seed(1)
    rnd = lambda *s: torch.randn(*s, generator=g, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    work = []
    for counts, N, K in (([7], 136, 128), ([30, 0, 200], 264, 136), ([300, 600], 512, 256)):
        rows, E = sum(counts), len(counts)
        off = None if E == 1 else torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32, device="cuda")
        a, w, dy = rnd(rows, K), rnd(E, N, K), rnd(rows, N)
        want = f32(rows, N), bf(rows, K), f32(E, N, K)
        got = [[torch.zeros_like(t) for t in want] for _ in range(20)]
        call = lambda o, s, a=a, w=w, dy=dy, off=off: (  # noqa: E731
            train.expert_linear(a, w, o[0], expert_offsets=off, stream=s),
            train.expert_linear_backward_input(dy, w, o[1], expert_offsets=off, stream=s),
            train.expert_linear_backward_weight(dy, a, o[2], expert_offsets=off, stream=s))
        call(want, None)
        work.append((call, want, got, torch.cuda.Stream()))
    torch.cuda.synchronize()
    start, errors = threading.Barrier(len(work)), []

    def go(call, got, stream):
        try:
            start.wait()
            for o in got:
                call(o, stream.cuda_stream)
        except Exception as e:  # noqa: BLE001
            errors.append(e)

    threads = [threading.Thread(target=go, args=(c, o, s)) for c, _, o, s in work]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not errors, errors
    for _, want, got, _ in work:
        for o in got:
            assert all(torch.equal(a, b) for a, b in zip(want, o))
