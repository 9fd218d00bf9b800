"""moe_router_topk and its gradient on the GPU against the formulas in 64 bits.

Indices are compared for equality.  Weights: exp and the quotients within 2 ulp,
the sums over E (or K) terms within their count of half steps."""
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

import train_ref as ref  # noqa: E402


@pytest.fixture(scope="module")
def train():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from combine_route_count_gb300 import build, moe, train as t
    build.build()
    build.build_train()
    moe.load_library()
    return t


GUARD = 64


def run(train, z, bias, K, score, normalize, scale, stream=None):
    T = z.shape[0]
    idx = torch.full((T * K + GUARD,), -7, dtype=torch.int32, device="cuda")
    w = torch.full((T * K + GUARD,), -7.0, device="cuda")
    train.router_topk(z, idx[: T * K].view(T, K), w[: T * K].view(T, K), score=score, bias=bias, normalize=normalize,
                      scale=scale, stream=stream)
    assert bool((idx[T * K:] == -7).all()) and bool((w[T * K:] == -7).all())
    return idx[: T * K].view(T, K), w[: T * K].view(T, K)


def error(E, z):
    """Relative error of a weight: exponents z - M and -z round to half a step of |z| each."""
    return (E / 8 + 24) * ref.F32 + 2 * z.abs().amax().item() * ref.F32


def check(train, z, bias, K, score, normalize, scale):
    idx, w = run(train, z, bias, K, score, normalize, scale)
    want = ref.choice(z.double(), None if bias is None else bias.double(), K)
    assert torch.equal(idx.long(), want)
    ww = ref.weights(z.double(), want, score, normalize, scale)
    assert bool(((w.double() - ww).abs() <= error(z.shape[1], z) * ww.abs() + 2.0 ** -126).all())
    return idx


def check_grad(train, z, idx, score, normalize, scale, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    T, E = z.shape
    dw = torch.randn(idx.shape, generator=g, device="cuda")
    d = torch.full((T * E + GUARD,), -7.0, dtype=z.dtype, device="cuda")
    train.router_topk_backward(z, idx, dw, d[: T * E].view(T, E), score=score, normalize=normalize, scale=scale)
    assert bool((d[T * E:] == -7).all())
    leaf = z.double().requires_grad_()
    out = ref.weights(leaf, idx.long(), score, normalize, scale)
    out.backward(dw.double())
    # Every term of the gradient is at most scale * |dw| * w; their sum over k bounds the differences.
    top = (dw.double().abs() * out.detach().abs()).sum(1, keepdim=True) + scale * 2.0 ** -100
    ref.near(d[: T * E].view(T, E), leaf.grad, 4 * (error(E, z) + 16 * ref.F32) * top)


@pytest.mark.parametrize("T,E,K", [(1, 1, 1), (1, 256, 8), (3, 2, 2), (5, 16, 16), (64, 8, 2), (129, 33, 5),
                                   (200, 384, 8), (31, 513, 16), (1030, 64, 6), (7, 1024, 16), (257, 40, 3)])
@pytest.mark.parametrize("score,bias,normalize", [("softmax", False, True), ("softmax", False, False),
                                                  ("sigmoid", False, True), ("sigmoid", True, True),
                                                  ("sigmoid", True, False)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_against_formula(train, T, E, K, score, bias, normalize, dtype):
    g = torch.Generator(device="cuda").manual_seed(T * 1000 + E)
    z = (2.0 * torch.randn(T, E, generator=g, device="cuda")).to(dtype)
    b = 0.2 * torch.randn(E, generator=g, device="cuda") if bias else None
    idx = check(train, z, b, K, score, normalize, 2.5)
    check_grad(train, z, idx, score, normalize, 2.5, E)


def test_equal_logits_take_the_lower_index(train):
    z = torch.zeros(33, 300, device="cuda")
    z[:, 7] = z[:, 250] = 1.0
    z[1::2, 100:200] = -0.0  # equal to 0
    idx = check(train, z, None, 8, "softmax", True, 1.0)
    assert idx[0].tolist() == [7, 250, 0, 1, 2, 3, 4, 5]
    idx = check(train, z, torch.zeros(300, device="cuda"), 8, "sigmoid", True, 1.0)
    assert idx[0].tolist() == [7, 250, 0, 1, 2, 3, 4, 5]


def test_sums_that_float32_cannot_tell_apart(train):
    """Keys sigmoid(z) + bias around 1/2 + 1/4, apart by 2^-30 at least: below float32's spacing there."""
    g = torch.Generator(device="cuda").manual_seed(5)
    T, E = 128, 256
    z = 0.001 * torch.randn(T, E, generator=g, device="cuda")
    b = (0.25 + 2.0 ** -27 * torch.randn(E, generator=g, device="cuda", dtype=torch.float64)).float()
    z[:, ::2] = torch.randint(-3, 4, (T, E // 2), generator=g, device="cuda").float() * 2.0 ** -26
    key = torch.sort(torch.sigmoid(z.double()) + b.double(), dim=1)[0]
    assert int((key.diff(dim=1) < 2.0 ** -25).sum()) > 1000
    check(train, z, b, 16, "sigmoid", True, 1.0)
    check(train, z, b - 1000.0, 16, "sigmoid", False, 1.0)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_masked_and_far_logits(train, score):
    g = torch.Generator(device="cuda").manual_seed(2)
    z = torch.randn(64, 48, generator=g, device="cuda")
    z[:, 5:] = -torch.inf          # fewer experts left than chosen: scores of zero
    z[1] = -torch.inf              # nothing left
    z[2] = -200.0 + torch.randn(48, generator=g, device="cuda")  # scores below float32's range
    z[3] = 80.0 + torch.randn(48, generator=g, device="cuda")
    z[4] = torch.finfo(torch.float32).min
    for normalize in (True, False):
        idx, w = run(train, z, None, 8, score, normalize, 1.0)
        want = ref.choice(z.double(), None, 8)
        assert torch.equal(idx.long(), want)
        assert bool((w[1] == 0).all()) and bool(torch.isfinite(w).all())
        ok = [i for i in range(64) if i not in (1, 4)]
        ww = ref.weights(z[ok].double(), want[ok], score, normalize, 1.0)
        rel = (12 + 48 / 8 + 24) * ref.F32 + 400 * ref.F32
        assert bool(((w[ok].double() - ww).abs() <= rel * ww + 2.0 ** -125).all())
        dw = torch.randn(64, 8, generator=g, device="cuda")
        d = torch.empty_like(z)
        train.router_topk_backward(z, idx, dw, d, score=score, normalize=normalize)
        assert bool(torch.isfinite(d).all()) and bool((d[1] == 0).all())
        assert bool((d[0, 5:] == 0).all())
    if score == "softmax":  # equal logits, however far down: equal weights
        idx, w = run(train, z, None, 8, score, True, 1.0)
        assert bool((w[4] == 0.125).all())


def test_nan_keeps_indices_apart(train):
    z = torch.randn(16, 100, device="cuda")
    z[0] = torch.nan
    z[1, 3] = torch.nan
    z[2, 4] = torch.inf
    z[3, ::2] = torch.nan
    for bias in (None, torch.randn(100, device="cuda")):
        idx, w = run(train, z, bias, 16, "sigmoid", True, 1.0)
        assert int(idx.min()) >= 0 and int(idx.max()) < 100
        s = idx.sort(1)[0]
        assert bool((s[:, 1:] > s[:, :-1]).all())
        assert torch.equal(idx[4:].long(), ref.choice(z[4:].double(), None if bias is None else bias.double(), 16))
        assert bool(torch.isfinite(w[4:]).all())


def test_gradient_against_differences(train):
    g = torch.Generator(device="cuda").manual_seed(9)
    for score, normalize in (("softmax", True), ("softmax", False), ("sigmoid", True), ("sigmoid", False)):
        z = torch.randn(6, 20, generator=g, device="cuda")
        dw = torch.randn(6, 4, generator=g, device="cuda")
        idx, _ = run(train, z, None, 4, score, normalize, 1.5)
        d = torch.empty_like(z)
        train.router_topk_backward(z, idx, dw, d, score=score, normalize=normalize, scale=1.5)
        h = 1e-5
        for e in range(20):
            up, down = z.double(), z.double()
            up[:, e] += h
            down[:, e] -= h
            slope = ((ref.weights(up, idx.long(), score, normalize, 1.5)
                      - ref.weights(down, idx.long(), score, normalize, 1.5)) * dw.double()).sum(1) / (2 * h)
            # third derivatives below 2: h^2 / 6 * 2 * |dw|, and float32's own error
            assert bool(((d[:, e].double() - slope).abs() <= 1e-5).all())


def test_indices_outside_and_twice(train):
    z = torch.randn(3, 10, device="cuda")
    dw = torch.randn(3, 3, device="cuda")
    for score in ("softmax", "sigmoid"):
        idx = torch.tensor([[1, -1, 2], [4, 4, 9], [10, 0, 1 << 30]], dtype=torch.int32, device="cuda")
        d = torch.empty_like(z)
        train.router_topk_backward(z, idx, dw, d, score=score, normalize=False)
        leaf = z.double().requires_grad_()
        p = ref.scores(leaf, score)
        out = sum((p[t, i] * dw[t, k].double() for t in range(3) for k, i in enumerate(idx[t].tolist()) if 0 <= i < 10))
        out.backward()
        assert bool(((d.double() - leaf.grad).abs() <= 64 * ref.F32 * (1 + dw.abs().max())).all())


def test_graph_and_other_stream(train):
    z = torch.randn(300, 96, device="cuda")
    idx = torch.empty(300, 4, dtype=torch.int32, device="cuda")
    w, dw, d = torch.empty(300, 4, device="cuda"), torch.randn(300, 4, device="cuda"), torch.empty_like(z)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    train.router_topk(z, idx, w, stream=side)
    side.synchronize()
    first = (idx.clone(), w.clone())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        train.router_topk(z, idx, w)
        train.router_topk_backward(z, idx, dw, d)
    z.copy_(torch.randn_like(z))
    graph.replay()
    torch.cuda.synchronize()
    again = torch.empty_like(idx), torch.empty_like(w)
    train.router_topk(z, *again)
    assert torch.equal(again[0], idx) and torch.equal(again[1], w) and not torch.equal(first[0], idx)
