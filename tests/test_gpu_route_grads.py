"""moe_combine_backward and moe_dispatch_backward on the GPU against the formulas in 64 bits.

Rows: one float32 product (or K - 1 sums) and one rounding to bf16; dot products
over H: a thread adds every 256th chunk in order, so that (H / 256 + 24) half
steps of the sum of magnitudes bound the error."""
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


def inputs(seed, T, H, K, extra=5):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rows = T * K + extra
    slot = torch.randperm(rows, generator=g, device="cuda")[: T * K].to(torch.int32).view(T, K)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
    return r(T, H), r(rows, H), torch.rand(T, K, generator=g, device="cuda"), slot


SIZES = [(1, 8, 1), (1, 7168, 8), (3, 16, 16), (64, 256, 2), (65, 1416, 3), (130, 4096, 2), (33, 520, 9), (17, 2064, 5),
         (4100, 64, 6), (9000, 8, 1)]


@pytest.mark.parametrize("T,H,K", SIZES)
def test_combine_backward(train, T, H, K):
    g, y, w, slot = inputs(T + H, T, H, K)
    dy = torch.full_like(y, -7.25)
    dw = torch.full((T + 1, K), -7.25, device="cuda")
    train.combine_backward(g, slot, w, dy, expert_y=y, d_topk_w=dw[:T])
    at = slot.flatten().long()
    want = (w.double()[..., None] * g.double()[:, None]).view(T * K, H)
    ref.near(dy[at], want, ref.F32 * want.abs())
    left = torch.ones(len(y), dtype=torch.bool, device="cuda")
    left[at] = False
    assert bool((dy[left] == -7.25).all()) and bool((dw[T] == -7.25).all())
    prod = g.double()[:, None] * y[at].view(T, K, H).double()
    ref.near(dw[:T], prod.sum(2), (H / 256 + 24) * ref.F32 * prod.abs().sum(2))
    # without the weights' gradient; and in place
    alone = torch.full_like(y, -7.25)
    train.combine_backward(g, slot, w, alone)
    assert torch.equal(alone, dy)
    dw2 = torch.empty(T, K, device="cuda")
    train.combine_backward(g, slot, w, y, expert_y=y, d_topk_w=dw2)
    assert torch.equal(y[at], dy[at]) and torch.equal(dw2, dw[:T])


@pytest.mark.parametrize("T,H,K", SIZES)
@pytest.mark.parametrize("add", [False, True])
def test_dispatch_backward(train, T, H, K, add):
    more, y, _, slot = inputs(T * 3 + H, T, H, K)
    out = torch.full((T + 1, H), -7.25, dtype=torch.bfloat16, device="cuda")
    train.dispatch_backward(y, slot, out[:T], add=more if add else None)
    parts = y[slot.flatten().long()].view(T, K, H).double()
    want, size = parts.sum(1), parts.abs().sum(1)
    if add:
        want, size = want + more.double(), size + more.double().abs()
    ref.near(out[:T], want, K * ref.F32 * size)
    assert bool((out[T] == -7.25).all())
    if add:
        train.dispatch_backward(y, slot, more, add=more)
        assert torch.equal(more, out[:T])


def test_rows_outside_are_left_out(train):
    """After a routing error slot_row holds -1; no entry leads outside the buffers."""
    g, y, w, slot = inputs(0, 20, 136, 4, extra=0)
    slot[3, 1], slot[4], slot[5, 0], slot[6, 2] = -1, -1, 80, 2 ** 31 - 1
    dy, dw = torch.full_like(y, -7.25), torch.full((20, 4), -7.25, device="cuda")
    train.combine_backward(g, slot, w, dy, expert_y=y, d_topk_w=dw)
    ok = (slot >= 0) & (slot < 80)
    assert bool((dw[~ok] == 0).all()) and bool((dw[ok] != -7.25).all())
    at = slot[ok].long()
    want = (w.double()[..., None] * g.double()[:, None])[ok]
    ref.near(dy[at], want, ref.F32 * want.abs())
    left = torch.ones(80, dtype=torch.bool, device="cuda")
    left[at] = False
    assert int(left.sum()) == 7 and bool((dy[left] == -7.25).all())
    dx = torch.full((20, 136), -7.25, dtype=torch.bfloat16, device="cuda")
    train.dispatch_backward(y, slot, dx)
    parts = torch.where(ok[..., None], y[slot.long().clamp(0, 79)].double(), 0.0)
    ref.near(dx, parts.sum(1), 4 * ref.F32 * parts.abs().sum(1))
    assert bool((dx[4] == 0).all())


def test_infinities_stay_in_their_token(train):
    g, y, w, slot = inputs(1, 12, 512, 3, extra=0)
    g[2, 7], y[slot[5, 1].item(), 9] = torch.inf, torch.nan
    dy, dw = torch.empty_like(y), torch.empty(12, 3, device="cuda")
    train.combine_backward(g, slot, w, dy, expert_y=y, d_topk_w=dw)
    bad = torch.zeros(12, 3, dtype=torch.bool, device="cuda")
    bad[2], bad[5, 1] = True, True
    assert bool(torch.isfinite(dw[~bad]).all()) and not bool(torch.isfinite(dw[bad]).any())
    rows = torch.ones(36, dtype=torch.bool, device="cuda")
    rows[slot[2].long()] = False
    assert bool(torch.isfinite(dy[rows].float()).all())


def test_no_tokens_and_int16_bits(train):
    e = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda")
    s = torch.empty(0, 2, dtype=torch.int32, device="cuda")
    train.combine_backward(e, s, torch.empty(0, 2, device="cuda"), e, expert_y=e, d_topk_w=torch.empty(0, 2, device="cuda"))
    train.dispatch_backward(e, s, e)
    _, y, _, slot = inputs(2, 9, 64, 2)
    a = torch.empty(9, 64, dtype=torch.bfloat16, device="cuda")
    b = torch.empty(9, 64, dtype=torch.int16, device="cuda")
    train.dispatch_backward(y, slot, a)
    train.dispatch_backward(y.view(torch.int16), slot, b)
    assert torch.equal(a.view(torch.int16), b)


def test_offsets_past_32_bits(train):
    """Rows beyond 4 GiB from the buffers' start."""
    H, K = 8192, 2
    rows = 2 ** 31 // H + 300
    y = torch.zeros(rows, H, dtype=torch.bfloat16, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(3)
    slot = torch.tensor([[0, rows - 1], [rows - 2, 1], [rows - 280, 5]], dtype=torch.int32, device="cuda")
    y[slot.flatten().long()] = torch.randn(6, H, generator=g, device="cuda").to(torch.bfloat16)
    d = torch.randn(3, H, generator=g, device="cuda").to(torch.bfloat16)
    w, dw = torch.rand(3, K, generator=g, device="cuda"), torch.empty(3, K, device="cuda")
    dx = torch.empty(3, H, dtype=torch.bfloat16, device="cuda")
    train.dispatch_backward(y, slot, dx)
    ref.near(dx, y[slot.flatten().long()].view(3, K, H).double().sum(1), 2.0 ** -20)
    dy = torch.zeros_like(y)
    train.combine_backward(d, slot, w, dy, expert_y=y, d_topk_w=dw)
    want = (w.double()[..., None] * d.double()[:, None]).view(6, H)
    ref.near(dy[slot.flatten().long()], want, ref.F32 * want.abs())
