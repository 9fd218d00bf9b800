"""The bf16 expert products and their gradients on the GPU against the formulas in 64 bits.

Tolerances: train_ref.product_error times the sum of magnitudes, carried through
bias, activation and residual, and one rounding to the output's type.  Products
of small integers are exact in float32 and compared bit for bit."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

import train_ref as ref  # noqa: E402

GUARD = 3


@pytest.fixture(scope="module")
def train():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from combine_route_count_gb300 import build, moe, train as t
    build.build()
    build.build_train()
    moe.load_library()
    return t


def bf(g, *shape, integers=False, scale=1.0):
    if integers:
        return torch.randint(-3, 4, shape, generator=g, device="cuda").to(torch.bfloat16)
    return (scale * torch.randn(shape, generator=g, device="cuda")).to(torch.bfloat16)


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def offsets_of(counts):
    return torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32, device="cuda")


def guarded(rows, n, dtype):
    """A buffer with guard rows on both sides, and its middle."""
    buf = torch.full((rows + 2 * GUARD, n), -7.25, dtype=dtype, device="cuda")
    return buf, buf[GUARD: GUARD + rows]


def untouched(buf):
    assert bool((buf[:GUARD] == -7.25).all()) and bool((buf[-GUARD:] == -7.25).all())


# (rows of each expert or rows, N, K)
SHAPES = [(1, 8, 8), (1, 256, 64), (3, 264, 72), (128, 256, 128), (129, 128, 200), (300, 1000, 520),
          ([0, 5, 0, 128, 1], 256, 136), ([130, 0, 0], 520, 64), ([1] * 40, 72, 328), ([257, 3, 64, 65], 768, 1032),
          ([0, 0], 64, 64), (2048, 512, 64),
          # pairs of CTAs over ragged groups; sums split over 2, 4 and 8 CTAs, of each product in turn; few rows
          ([300, 0, 700, 513], 264, 136), (600, 1032, 1544), (600, 1544, 1032), (600, 520, 6152), (16400, 72, 72),
          (20, 264, 1032)]


def split(shape):
    counts, N, K = shape
    if isinstance(counts, int):
        return counts, 1, N, K, None
    return sum(counts), len(counts), N, K, offsets_of(counts)


@pytest.mark.parametrize("shape", SHAPES)
def test_integers_are_exact(train, shape):
    rows, E, N, K, off = split(shape)
    g = gen(rows + N + K)
    a, w, dy = bf(g, rows, K, integers=True), bf(g, E, N, K, integers=True), bf(g, rows, N, integers=True)
    buf, out = guarded(rows, N, torch.float32)
    train.expert_linear(a, w, out, expert_offsets=off)
    assert torch.equal(out.double(), ref.forward(a, w, off)[0])
    untouched(buf)
    buf, dx = guarded(rows, K, torch.bfloat16)
    train.expert_linear_backward_input(dy, w, dx, expert_offsets=off)
    assert torch.equal(dx, ref.by_rows(dy, w, off)[0].to(torch.bfloat16))
    untouched(buf)
    wbuf, dw = guarded(E * N, K, torch.float32)
    store = torch.full((E * N + 8,), -7.25, device="cuda")
    db = store[4: 4 + E * N].view(E, N)
    train.expert_linear_backward_weight(dy, a, dw.view(E, N, K), db=db, expert_offsets=off)
    want, _, want_b, _ = ref.by_weights(dy, a, off, E)
    assert torch.equal(dw.view(E, N, K).double(), want) and torch.equal(db.double(), want_b)
    assert bool((store[:4] == -7.25).all()) and bool((store[4 + E * N:] == -7.25).all())
    untouched(wbuf)


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("activation", ["none", "relu", "gelu", "silu", "swiglu"])
@pytest.mark.parametrize("out_type", [torch.bfloat16, torch.float32])
def test_forward_epilogue(train, shape, activation, out_type):
    rows, E, N, K, off = split(shape)
    glu = activation == "swiglu"
    if glu:
        N *= 2
    n_out = N // 2 if glu else N
    g = gen(rows * 3 + N + K)
    a, w = bf(g, rows, K), bf(g, E, N, K, scale=2.0 / K ** 0.5)
    for bias_type, residual, with_pre in ((None, False, False), (torch.bfloat16, True, True), (torch.float32, False, True),
                                          (torch.float32, True, False)):
        bias = None if bias_type is None else torch.randn(E, N, generator=g, device="cuda").to(bias_type)
        res = bf(g, rows, n_out) if residual else None
        buf, out = guarded(rows, n_out, out_type)
        pbuf, pre = guarded(rows, N, torch.bfloat16)
        train.expert_linear(a, w, out, bias=bias, activation=activation, residual=res, pre=pre if with_pre else None,
                            expert_offsets=off)
        v, s = ref.forward(a, w, off)
        err = ref.product_error(K) * s
        if bias is not None:
            for e, (lo, hi) in enumerate(ref.clamped(off, rows, E)):
                v[lo:hi] += bias[e].double()
            err = err + ref.F32 * (v.abs() + err)
        if with_pre:
            ref.near(pre, v, err)
        h, herr = ref.act(activation, v), ref.act_error(activation, v, err)
        if residual:
            h = h + res.double()
            herr = herr + ref.F32 * (h.abs() + herr)
        ref.near(out, h, herr)
        untouched(buf)
        untouched(pbuf)


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("activation", ["none", "relu", "gelu", "silu", "swiglu"])
def test_backward_input(train, shape, activation):
    rows, E, N, K, off = split(shape)
    wide = 2 * K if activation == "swiglu" else K
    g = gen(rows * 5 + N + K)
    dy, w = bf(g, rows, N), bf(g, E, N, K, scale=1.0 / N ** 0.5)
    pre = None if activation == "none" else bf(g, rows, wide, scale=2.0)
    buf, dx = guarded(rows, wide, torch.bfloat16)
    train.expert_linear_backward_input(dy, w, dx, activation=activation, pre=pre, expert_offsets=off)
    v, s = ref.by_rows(dy, w, off)
    d, err = ref.through(activation, v, ref.product_error(N) * s, None if pre is None else pre.double())
    ref.near(dx, d, err)
    untouched(buf)
    if pre is not None:  # in place
        train.expert_linear_backward_input(dy, w, pre, activation=activation, pre=pre, expert_offsets=off)
        assert torch.equal(pre, dx)


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_backward_weight(train, shape, dtype):
    rows, E, N, K, off = split(shape)
    g = gen(rows * 7 + N + K)
    dy, a = bf(g, rows, N), bf(g, rows, K)
    dw = torch.full((E, N, K), -7.25, dtype=dtype, device="cuda")
    db = torch.full((E, N), -7.25, device="cuda")
    train.expert_linear_backward_weight(dy, a, dw, db=db, expert_offsets=off)
    most = max([hi - lo for lo, hi in ref.clamped(off, rows, E)])
    want, s, want_b, sb = ref.by_weights(dy, a, off, E)
    ref.near(dw, want, ref.product_error(most) * s)
    ref.near(db, want_b, (most + 1) * ref.F32 * sb)
    alone = torch.empty_like(dw)
    train.expert_linear_backward_weight(dy, a, alone, expert_offsets=off)
    assert torch.equal(alone, dw)
    old, old_b = dw.double(), db.double()
    train.expert_linear_backward_weight(dy, a, dw, db=db, accumulate=True, expert_offsets=off)
    ref.near(dw, want + old, ref.product_error(most) * s + ref.F32 * (want + old).abs())
    ref.near(db, want_b + old_b, (most + 2) * ref.F32 * sb + ref.F32 * old_b.abs())


def test_rows_and_experts_without_an_owner(train):
    """Damaged offsets are clamped; rows that no expert owns are left untouched.  Where
    they decrease, a row may have two owners: out holds either's product."""
    g = gen(0)
    a, w, dy = bf(g, 50, 64, integers=True), bf(g, 4, 72, 64, integers=True), bf(g, 50, 72, integers=True)
    for off in ([5, 9, 9, 30, 40], [-100, 7, 3, 2 ** 31 - 1, 2 ** 31 - 1], [60, 70, 80, 90, 100], [0, 0, 0, 0, 0]):
        offsets = torch.tensor(off, dtype=torch.int32, device="cuda")
        owners = torch.zeros(50, dtype=torch.int32, device="cuda")
        for lo, hi in ref.clamped(off, 50, 4):
            owners[lo:hi] += 1
        once, none = owners == 1, owners == 0
        out = torch.full((50, 72), -7.25, device="cuda")
        train.expert_linear(a, w, out, expert_offsets=offsets)
        want = ref.forward(a, w, off)[0]
        assert torch.equal(out[once].double(), want[once]) and bool((out[none] == -7.25).all())
        dw, db = torch.empty(4, 72, 64, device="cuda"), torch.empty(4, 72, device="cuda")
        train.expert_linear_backward_weight(dy, a, dw, db=db, expert_offsets=offsets)
        want, _, want_b, _ = ref.by_weights(dy, a, off, 4)
        assert torch.equal(dw.double(), want) and torch.equal(db.double(), want_b)


def test_infinities_stay_in_their_rows_and_experts(train):
    g = gen(1)
    counts, N, K = [20, 33, 70], 136, 72
    off = offsets_of(counts)
    a, w, dy = bf(g, 123, K), bf(g, 3, N, K), bf(g, 123, N)
    a[20 + 5], w[0, 3], dy[53] = torch.inf, torch.nan, torch.nan
    out = torch.empty(123, N, device="cuda")
    train.expert_linear(a, w, out, expert_offsets=off)
    ok = torch.ones(123, N, dtype=torch.bool, device="cuda")
    ok[25], ok[:20, 3] = False, False
    assert bool(torch.isfinite(out[ok]).all()) and not bool(torch.isfinite(out[~ok]).any())
    dx = torch.empty(123, K, dtype=torch.bfloat16, device="cuda")
    train.expert_linear_backward_input(dy, w, dx, expert_offsets=off)
    fine = torch.isfinite(dx.float()).all(1)
    assert not bool(fine[:20].any()) and not bool(fine[53]) and bool(fine[20:53].all()) and bool(fine[54:].all())
    dw, db = torch.empty(3, N, K, device="cuda"), torch.empty(3, N, device="cuda")
    train.expert_linear_backward_weight(dy, a, dw, db=db, expert_offsets=off)
    assert bool(torch.isfinite(dw[0]).all()) and not bool(torch.isfinite(dw[1]).any()) and not bool(torch.isfinite(dw[2]).any())
    assert bool(torch.isfinite(db[:2]).all()) and not bool(torch.isfinite(db[2]).any())


def test_no_rows(train):
    off = torch.zeros(3, dtype=torch.int32, device="cuda")
    e = lambda n: torch.empty(0, n, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    w = torch.zeros(2, 16, 8, dtype=torch.bfloat16, device="cuda")
    train.expert_linear(e(8), w, e(16), expert_offsets=off)
    train.expert_linear_backward_input(e(16), w, e(8), expert_offsets=off)
    dw, db = torch.ones(2, 16, 8, device="cuda"), torch.ones(2, 16, device="cuda")
    train.expert_linear_backward_weight(e(16), e(8), dw, db=db, accumulate=True, expert_offsets=off)
    assert bool((dw == 1).all()) and bool((db == 1).all())
    train.expert_linear_backward_weight(e(16), e(8), dw, db=db, expert_offsets=off)
    assert bool((dw == 0).all()) and bool((db == 0).all())


def test_residual_in_place_and_one_matrix(train):
    g = gen(4)
    a, w, r = bf(g, 77, 128), bf(g, 200, 128), bf(g, 77, 200)
    out = torch.empty_like(r)
    train.expert_linear(a, w, out, residual=r)
    train.expert_linear(a, w, r, residual=r)
    assert torch.equal(out, r)


def test_graph_replay_and_streams(train):
    g = gen(6)
    counts = [40, 0, 300, 7]
    a, w, off = bf(g, 347, 192), bf(g, 4, 320, 192), offsets_of(counts)
    dy = bf(g, 347, 320)
    out, dx = torch.empty(347, 320, device="cuda"), torch.empty(347, 192, dtype=torch.bfloat16, device="cuda")
    dw = torch.empty(4, 320, 192, device="cuda")

    def calls(stream=None):
        train.expert_linear(a, w, out, expert_offsets=off, stream=stream)
        train.expert_linear_backward_input(dy, w, dx, expert_offsets=off, stream=stream)
        train.expert_linear_backward_weight(dy, a, dw, expert_offsets=off, stream=stream)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    calls(side)
    side.synchronize()
    first = [t.clone() for t in (out, dx, dw)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        calls()
    for t in (out, dx, dw):
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(first, (out, dx, dw)))
    off.copy_(offsets_of([1, 100, 46, 200]))  # read on the device at each replay
    graph.replay()
    torch.cuda.synchronize()
    again = torch.empty_like(out)
    train.expert_linear(a, w, again, expert_offsets=off)
    assert torch.equal(again, out) and not torch.equal(again, first[0])


def test_offsets_past_32_bits(train):
    """Weights, gradients and rows beyond 2^31 elements from their buffers' start."""
    g = gen(8)
    E, N, K = 70, 8192, 4096
    w = torch.zeros(E, N, K, dtype=torch.bfloat16, device="cuda")
    w[69, -64:] = bf(g, 64, K, integers=True)
    for rows in (8, 900):  # few rows, and tiles
        counts = [3] + [0] * 68 + [rows - 3]
        off = offsets_of(counts)
        a, dy = bf(g, rows, K, integers=True), torch.zeros(rows, N, dtype=torch.bfloat16, device="cuda")
        dy[:, -64:] = bf(g, rows, 64, integers=True)
        out = torch.full((rows, N), -7.25, device="cuda")
        train.expert_linear(a, w, out, expert_offsets=off)
        assert torch.equal(out[3:, -64:].double(), a[3:].double() @ w[69, -64:].double().t())
        assert not bool(out[:3].any()) and not bool(out[3:, :-64].any())
        dx = torch.empty(rows, K, dtype=torch.bfloat16, device="cuda")
        train.expert_linear_backward_input(dy, w, dx, expert_offsets=off)
        assert torch.equal(dx[3:], (dy[3:, -64:].double() @ w[69, -64:].double()).to(torch.bfloat16))
        assert not bool(dx[:3].any())
        dw = torch.full_like(w, -7.25)
        train.expert_linear_backward_weight(dy, a, dw, expert_offsets=off)
        assert torch.equal(dw[69, -64:], (dy[3:, -64:].double().t() @ a[3:].double()).to(torch.bfloat16))
        assert not bool(dw[1:69].any()) and not bool(dw[69, :-64].any())
    del w, dw
    rows, N, K = 2 ** 31 // 8192 + 300, 8192, 64
    a, w = bf(g, rows, K, integers=True), bf(g, N, K, integers=True)
    r = torch.zeros(rows, N, dtype=torch.bfloat16, device="cuda")
    r[-400:] = 1.0
    train.expert_linear(a, w, r, residual=r)
    want = a[-400:].double() @ w.double().t() + 1.0
    assert torch.equal(r[-400:], want.to(torch.bfloat16))
    assert torch.equal(r[:10], (a[:10].double() @ w.double().t()).to(torch.bfloat16))


def test_many_shapes(train):
    """Shapes over the range in which a call changes its kernel, all three products of each."""
    import random
    rng = random.Random(12)
    size = lambda hi: 8 * max(1, int(2 ** rng.uniform(0, np.log2(hi / 8))))  # noqa: E731
    for i in range(60):
        g = gen(1000 + i)
        E = rng.choice([1, 1, 2, 5, 40])
        N, K, rows = size(1200), size(2000), int(2 ** rng.uniform(0, 11))
        cuts = sorted(rng.randint(0, rows) for _ in range(E - 1))
        off = None if E == 1 else torch.tensor([0, *cuts, rows], dtype=torch.int32, device="cuda")
        a, w, dy = bf(g, rows, K, integers=True), bf(g, E, N, K, integers=True), bf(g, rows, N, integers=True)
        out, dx = torch.empty(rows, N, device="cuda"), torch.empty(rows, K, dtype=torch.bfloat16, device="cuda")
        dw, db = torch.empty(E, N, K, device="cuda"), torch.empty(E, N, device="cuda")
        train.expert_linear(a, w, out, expert_offsets=off)
        train.expert_linear_backward_input(dy, w, dx, expert_offsets=off)
        train.expert_linear_backward_weight(dy, a, dw, db=db, expert_offsets=off)
        want, _, want_b, _ = ref.by_weights(dy, a, off, E)
        assert torch.equal(out.double(), ref.forward(a, w, off)[0]), (rows, E, N, K)
        assert torch.equal(dx, ref.by_rows(dy, w, off)[0].to(torch.bfloat16)), (rows, E, N, K)
        assert torch.equal(dw.double(), want) and torch.equal(db.double(), want_b), (rows, E, N, K)
