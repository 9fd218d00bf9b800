"""moe_decode_layer_fp8 on the GPU against the layer in 64 bits (ffn_ref.decode_layer and its bound)."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

import ffn_ref as ref  # noqa: E402


@pytest.fixture(scope="module")
def ffn():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from combine_route_count_gb300 import build, ffn as f, moe
    build.build()
    build.build_ffn()
    moe.load_library()
    return f


def codes(g, *shape):
    return (torch.randn(shape, generator=g, device="cuda") * 100).clamp(-448, 448).to(torch.float8_e4m3fn)


def scales(g, *shape):
    return 0.0005 + torch.rand(shape, generator=g, device="cuda") * 0.001


def weights(seed, E, H, I):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return codes(g, E, 2 * I, H), scales(g, E, 2 * I // 128, H // 128), codes(g, E, H, I), scales(g, E, H // 128, I // 128)


def tokens(seed, T, H, K, E, hot=False):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rng = np.random.default_rng(seed)
    idx = np.stack([rng.permutation(K) if hot else rng.permutation(E)[:K] for _ in range(T)]).astype(np.int32)
    w = torch.softmax(torch.randn(T, K, generator=g, device="cuda"), 1)
    return codes(g, T, H), scales(g, T, H // 128), torch.from_numpy(idx).cuda(), w


def run(layer, x, sx, idx, w, stream=None):
    T, H = x.shape
    buf = torch.full((T + 2, H), -7.25, dtype=torch.bfloat16, device="cuda")
    torch.cuda.synchronize()
    layer.forward(x, sx, idx, w, buf[1:1 + T], stream=stream)
    assert layer.get_error(stream) == 0
    assert (buf[0] == -7.25).all() and (buf[-1] == -7.25).all()
    return buf[1:1 + T]


def check(ffn, T, H, I, E, K, hot=False):
    ws, tk = weights(T + H, E, H, I), tokens(T * 31 + I, T, H, K, E, hot)
    out = run(ffn.DecodeLayer(T, K, *ws), *tk)
    want, bound = ref.decode_layer(*tk, *ws)
    far = (out.double() - want).abs() - bound
    assert (far <= 0).all(), float(far.max())
    # The bound takes every code that may fall either way at its worst; over
    # the whole output, rounding to bf16 (0.2 percent) has to be what is left.
    assert float((out.double() - want).norm()) < 0.005 * float(want.norm())


@pytest.mark.parametrize("T", [1, 2, 7, 8, 9, 16, 17, 32, 33, 64])
@pytest.mark.parametrize("H,I,E,K", [(256, 512, 8, 2), (128, 128, 1, 1), (1152, 384, 40, 6), (512, 1408, 5, 5)])
def test_sizes(ffn, T, H, I, E, K):
    check(ffn, T, H, I, E, K)


@pytest.mark.parametrize("T", [1, 13, 40, 64])
def test_every_token_on_the_same_experts(ffn, T):
    check(ffn, T, 640, 256, 32, 3, hot=True)


def test_many_experts_and_choices(ffn):
    check(ffn, 64, 256, 128, 1024, 16)
    check(ffn, 1, 256, 128, 1024, 16)


@pytest.mark.parametrize("T", [1, 24])
def test_long_rows(ffn, T):
    check(ffn, T, 7168, 2048, 12, 4)


def test_one_layer_object_for_every_batch_size(ffn):
    ws = weights(3, 16, 512, 256)
    layer = ffn.DecodeLayer(64, 4, *ws)
    for T in (64, 1, 30, 5, 64, 2):
        tk = tokens(T, T, 512, 4, 16)
        want, bound = ref.decode_layer(*tk, *ws)
        assert ((run(layer, *tk).double() - want).abs() <= bound).all()


def test_no_tokens(ffn):
    layer = ffn.DecodeLayer(4, 2, *weights(4, 4, 256, 128))
    layer.forward(torch.empty(0, 256, dtype=torch.uint8, device="cuda"), torch.empty(0, 2, device="cuda"),
                  torch.empty(0, 2, dtype=torch.int32, device="cuda"), torch.empty(0, 2, device="cuda"),
                  torch.empty(0, 256, dtype=torch.bfloat16, device="cuda"))


@pytest.mark.parametrize("bad", ["high", "negative", "repeated"])
@pytest.mark.parametrize("T", [1, 40])
def test_bad_routing_writes_nothing(ffn, bad, T):
    from combine_route_count_gb300 import moe
    ws = weights(5, 8, 256, 128)
    layer = ffn.DecodeLayer(64, 3, *ws)
    x, sx, idx, w = tokens(6, T, 256, 3, 8)
    wrong = idx.clone()
    wrong[T - 1, 2] = {"high": 8, "negative": -1, "repeated": int(idx[T - 1, 0])}[bad]
    out = torch.full((T, 256), -7.25, dtype=torch.bfloat16, device="cuda")
    layer.forward(x, sx, wrong, w, out)
    assert layer.get_error() == moe.MOE_EROUTE
    assert (out == -7.25).all()
    want, bound = ref.decode_layer(x, sx, idx, w, *ws)
    assert ((run(layer, x, sx, idx, w).double() - want).abs() <= bound).all()


def test_special_values(ffn):
    """A token of zeros gives zeros; a NaN scale stays in its token; saturated gates stay finite."""
    ws = weights(7, 8, 256, 128)
    x, sx, idx, w = tokens(8, 20, 256, 2, 8)
    x.view(torch.uint8)[3] = 0
    sx[7, 1] = float("nan")
    sx[11] *= 1e6
    out = run(ffn.DecodeLayer(20, 2, *ws), x, sx, idx, w).double()
    good = [t for t in range(20) if t not in (7, 11)]
    want, bound = ref.decode_layer(x[good], sx[good], idx[good], w[good], *ws)
    assert ((out[good] - want).abs() <= bound).all()
    assert (out[3] == 0).all() and torch.isfinite(out[11]).all()


def test_same_result_every_time_and_on_another_stream(ffn):
    ws = weights(9, 16, 512, 384)
    for T in (3, 50):
        tk = tokens(10, T, 512, 4, 16)
        layer = ffn.DecodeLayer(64, 4, *ws)
        a = run(layer, *tk)
        assert torch.equal(a, run(layer, *tk)) and torch.equal(a, run(layer, *tk, stream=torch.cuda.Stream()))


def test_back_to_back_calls_and_graphs(ffn):
    """Calls in a row share the workspace: each must see its own h, in a stream and in a graph."""
    ws = weights(11, 16, 512, 384)
    layer = ffn.DecodeLayer(32, 4, *ws)
    batches = [tokens(20 + i, T, 512, 4, 16) for i, T in enumerate((32, 1, 17, 8, 25))]
    alone = [run(layer, *b) for b in batches]
    outs = [torch.empty_like(a) for a in alone]

    def all_of_them():
        for b, o in zip(batches, outs):
            layer.forward(*b, o)

    for _ in range(20):
        all_of_them()
    torch.cuda.synchronize()
    assert all(torch.equal(a, o) for a, o in zip(alone, outs))
    for o in outs:
        o.zero_()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        all_of_them()
    for _ in range(5):
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, o) for a, o in zip(alone, outs))


def test_agrees_with_the_dispatched_layer(ffn):
    """Dispatch, both products and combine give the same layer, but for expert_y's rounding to bf16."""
    from combine_route_count_gb300 import moe
    T, H, I, E, K = 48, 512, 256, 16, 4
    ws, tk = weights(12, E, H, I), tokens(13, T, H, K, E)
    x, sx, idx, w = tk
    layer = moe.MoELayer(T, H, K, E, 1)
    rows = T * K
    ex, es = torch.empty(rows, H, dtype=torch.uint8, device="cuda"), torch.empty(rows, H // 128, device="cuda")
    layer.dispatch_send_quantized(x, sx, idx, ex, es)
    lay = layer.dispatch_recv()
    hq, hs = torch.empty(rows, I, dtype=torch.uint8, device="cuda"), torch.empty(rows, I // 128, device="cuda")
    ffn.expert_glu_fp8(ex, es, ws[0], ws[1], hq, hs, expert_offsets=lay["expert_offsets"])
    y = torch.empty(rows, H, dtype=torch.bfloat16, device="cuda")
    ffn.expert_gemm_fp8(hq, hs, ws[2], ws[3], y, expert_offsets=lay["expert_offsets"])
    layer.combine_send(y)
    out = torch.empty(T, H, dtype=torch.bfloat16, device="cuda")
    layer.combine_recv(w, out)
    assert layer.get_error() == 0
    want, bound = ref.decode_layer(*tk, *ws)
    slot = lay["slot_row"].long()
    bound = bound + 2.0 ** -8 * (w[..., None].double() * y[slot].double().abs()).sum(1)
    assert ((out.double() - want).abs() <= bound).all()
    assert ((run(ffn.DecodeLayer(T, K, *ws), *tk).double() - want).abs() <= bound).all()


def test_refusals(ffn):
    from combine_route_count_gb300 import moe
    ws = weights(14, 8, 256, 128)
    for args in [(65, 2, *ws), (-1, 2, *ws), (4, 9, *ws), (4, 17, *ws), (4, 2, ws[0][:, :128].contiguous(), *ws[1:]),
                 (4, 2, ws[0], ws[1][:4], *ws[2:]), (4, 2, ws[0].float(), *ws[1:]), (4, 2, ws[0], ws[1], ws[2].cpu(), ws[3])]:
        with pytest.raises(moe.MoEError) as e:
            ffn.DecodeLayer(*args)
        assert e.value.code == moe.MOE_EINVAL
    layer = ffn.DecodeLayer(4, 2, *ws)
    x, sx, idx, w = tokens(15, 4, 256, 2, 8)
    out = torch.zeros(4, 256, dtype=torch.bfloat16, device="cuda")
    five = tokens(15, 5, 256, 2, 8)
    for args in [(*five, out), (x, sx, idx.long(), w, out), (x, sx, idx, w.double(), out), (x, sx[:, :1], idx, w, out),
                 (x, sx, idx[:, :1], w, out), (x, sx, idx, w, out.float()), (x.t(), sx, idx, w, out),
                 (x, sx, idx, w, out[:, ::2])]:
        with pytest.raises(moe.MoEError) as e:
            layer.forward(*args)
        assert e.value.code == moe.MOE_EINVAL
    assert (out == 0).all()
