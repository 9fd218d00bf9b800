"""moe_expert_gemm_fp8 and moe_expert_glu_fp8 on the GPU against the formulas in 64 bits.

Tolerances: ffn_ref.product_error times the sum of magnitudes for float32
outputs, plus half a bf16 step for bf16 ones; for the quantised h the bound of
ffn_ref.glu, then half a code step.  Products of small integers with scales
that are powers of two are exact in float32 and compared bit for bit."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

import ffn_ref as ref  # noqa: E402

GUARD = 3


@pytest.fixture(scope="module")
def ffn():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from combine_route_count_gb300 import build, ffn as f, moe
    build.build()
    build.build_ffn()
    moe.load_library()
    return f


def blocks(n):
    return -(-n // 128)


def codes(g, *shape, integers=False):
    if integers:
        return torch.randint(-4, 5, shape, generator=g, device="cuda").float().to(torch.float8_e4m3fn)
    return (torch.randn(shape, generator=g, device="cuda") * 100).clamp(-448, 448).to(torch.float8_e4m3fn)


def scales(g, *shape, integers=False):
    if integers:
        return torch.exp2(torch.randint(-2, 3, shape, generator=g, device="cuda").float())
    return 0.001 + torch.rand(shape, generator=g, device="cuda") * 0.01


def inputs(seed, rows, E, N, K, integers=False):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (codes(g, rows, K, integers=integers), scales(g, rows, blocks(K), integers=integers),
            codes(g, E, N, K, integers=integers), scales(g, E, blocks(N), blocks(K), integers=integers))


def offsets_of(counts):
    return torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32, device="cuda")


def gemm(ffn, a, sa, w, sw, off, dtype, stream=None):
    rows, N = a.shape[0], w.shape[-2]
    buf = torch.full((rows + 2 * GUARD, N), -7.25, dtype=dtype, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    ffn.expert_gemm_fp8(a, sa, w, sw, buf[GUARD:GUARD + rows], expert_offsets=off, status=status, stream=stream)
    torch.cuda.synchronize()
    assert int(status) == 0
    assert (buf[:GUARD] == -7.25).all() and (buf[GUARD + rows:] == -7.25).all()
    return buf[GUARD:GUARD + rows]


def check_gemm(ffn, a, sa, w, sw, off, dtype, exact=False):
    out = gemm(ffn, a, sa, w, sw, off, dtype).double()
    P, S = ref.product(a, sa, w, sw, None if off is None else off.tolist())
    if exact:
        assert torch.equal(out, P)
        return
    tol = ref.product_error(sa.shape[1]) * S
    if dtype == torch.bfloat16:
        _, e = torch.frexp(P.abs() + tol)
        tol = tol + torch.exp2(e.double() - 9)
    far = (out - P).abs() - tol
    assert (far <= 0).all(), float(far.max())


def glu(ffn, a, sa, w, sw, off, stream=None):
    rows, I = a.shape[0], w.shape[-2] // 2
    q = torch.full((rows + 2 * GUARD, I), 0x5A, dtype=torch.uint8, device="cuda")
    s = torch.full((rows + 2 * GUARD, I // 128), -7.25, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    ffn.expert_glu_fp8(a, sa, w, sw, q[GUARD:GUARD + rows], s[GUARD:GUARD + rows], expert_offsets=off, status=status,
                       stream=stream)
    torch.cuda.synchronize()
    assert int(status) == 0
    for edge in (slice(0, GUARD), slice(GUARD + rows, None)):
        assert (q[edge] == 0x5A).all() and (s[edge] == -7.25).all()
    return q[GUARD:GUARD + rows], s[GUARD:GUARD + rows]


def check_glu(ffn, a, sa, w, sw, off):
    q, s = glu(ffn, a, sa, w, sw, off)
    P, S = ref.product(a, sa, w, sw, None if off is None else off.tolist())
    h, err = ref.glu(P, S, ref.product_error(sa.shape[1]))
    shape = (h.shape[0], -1, 128)
    top = h.abs().view(shape).amax(-1)
    rel = err.view(shape).amax(-1) / top.clamp_min(1e-300)
    ref.assert_codes_near(ref.f64(q.view(torch.float8_e4m3fn).float()), ref.f64(s), ref.f64(h), ref.f64(rel) + 2.0 ** -22)


@pytest.mark.parametrize("rows", [1, 2, 8, 9, 33, 64, 65, 127, 128, 129, 300])
@pytest.mark.parametrize("N,K", [(8, 16), (128, 128), (264, 400), (512, 1024), (1416, 2320)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_dense(ffn, rows, N, K, dtype):
    check_gemm(ffn, *inputs(rows + N, rows, 1, N, K), None, dtype)


COUNTS = {
    "even": [5] * 16,
    "ragged": [0, 1, 130, 0, 7, 128, 64, 0, 0, 257, 3],
    "one_hot": [0, 0, 0, 700, 0],
    "ones": [1] * 70,
    "many": [(7 * i * i) % 5 for i in range(1024)],
    "empty": [0] * 9,
}


@pytest.mark.parametrize("name", list(COUNTS))
@pytest.mark.parametrize("N,K", [(136, 144), (384, 512)])
@pytest.mark.parametrize("exact", [True, False])
def test_grouped(ffn, name, N, K, exact):
    counts = COUNTS[name]
    rows = max(sum(counts), 4)
    args = inputs(len(counts), rows, len(counts), N, K, integers=exact)
    off = offsets_of(counts)
    if sum(counts) == 0:
        assert (gemm(ffn, *args, off, torch.float32) == -7.25).all()
        return
    check_gemm(ffn, *args, off, torch.float32, exact)
    check_gemm(ffn, *args, off, torch.bfloat16)


@pytest.mark.parametrize("name", ["even", "ragged", "one_hot", "ones"])
@pytest.mark.parametrize("I,H", [(128, 128), (256, 400), (640, 1024), (128, 7168)])
def test_glu(ffn, name, I, H):
    counts = COUNTS[name]
    check_glu(ffn, *inputs(I + H, sum(counts), len(counts), 2 * I, H), offsets_of(counts))


@pytest.mark.parametrize("rows", [1, 5, 17, 64, 100, 128, 200, 1000])
def test_glu_dense(ffn, rows):
    check_glu(ffn, *inputs(rows, rows, 1, 2 * 384, 640), None)


def test_more_tiles_than_sms(ffn):
    counts = [40, 300, 0, 129, 500, 16, 128, 256]
    check_gemm(ffn, *inputs(1, sum(counts), 8, 7168, 256), offsets_of(counts), torch.bfloat16)
    check_glu(ffn, *inputs(2, sum(counts), 8, 2 * 4096, 256), offsets_of(counts))


def test_long_k(ffn):
    check_gemm(ffn, *inputs(3, 130, 1, 256, 65536), None, torch.float32)
    check_gemm(ffn, *inputs(3, 6, 1, 256, 65536), None, torch.float32)


# K long enough that products of few rows are split along it, and kernels that
# put weight rows into the matrix tile take over; with a last block of 16.
@pytest.mark.parametrize("name", ["even", "ragged", "ones", "many", "one_hot"])
@pytest.mark.parametrize("N", [8, 264, 640])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_grouped_long_k(ffn, name, N, dtype):
    counts = COUNTS[name]
    check_gemm(ffn, *inputs(N, sum(counts), len(counts), N, 25 * 128 + 16 if name == "many" else 40 * 128 + 16),
               offsets_of(counts), dtype)


@pytest.mark.parametrize("rows", [1, 16, 17, 32, 33, 64, 100, 128, 129])
@pytest.mark.parametrize("N,K", [(1024, 6000), (136, 4096), (24, 26 * 128)])
def test_dense_long_k(ffn, rows, N, K):
    check_gemm(ffn, *inputs(rows, rows, 1, N, K), None, torch.float32)
    check_gemm(ffn, *inputs(rows, rows, 1, N, K, integers=True), None, torch.float32, exact=K < 4096)


@pytest.mark.parametrize("rows_each", [1, 2, 15, 16, 17, 40, 64, 65, 130])
def test_glu_rows_per_expert(ffn, rows_each):
    """Across the sizes at which another kernel takes over, with one expert far fuller than the others."""
    counts = [rows_each] * 12
    counts[3], counts[7] = 0, 3 * rows_each
    check_glu(ffn, *inputs(rows_each, sum(counts), 12, 2 * 1024, 768), offsets_of(counts))
    check_glu(ffn, *inputs(rows_each, sum(counts), 12, 2 * 256, 768), offsets_of(counts))


def test_glu_many_experts(ffn):
    counts = [(5 * i) % 7 for i in range(1024)]
    check_glu(ffn, *inputs(1, sum(counts), 1024, 2 * 128, 256), offsets_of(counts))


def test_rows_that_no_expert_owns_stay(ffn):
    for off in ([3, 5, 5, 9], [4, 4, 4, 4]):
        a, sa, w, sw = inputs(4, 12, 3, 128, 128, integers=True)
        out = gemm(ffn, a, sa, w, sw, torch.tensor(off, dtype=torch.int32, device="cuda"), torch.float32)
        P, _ = ref.product(a, sa, w, sw, off)
        assert torch.equal(out[off[0]:off[-1]].double(), P[off[0]:off[-1]])
        assert (out[:off[0]] == -7.25).all() and (out[off[-1]:] == -7.25).all()


@pytest.mark.parametrize("off", [[-5, 4, 8, 12], [0, 4, 400, 12], [0, 2 ** 31 - 1, -2 ** 31, 7], [9, 3, 1, 0]])
def test_damaged_offsets_stay_inside(ffn, off):
    """Offsets out of order or out of range write nothing outside the rows (the guard rows tell)."""
    a, sa, w, sw = inputs(5, 12, 3, 256, 256)
    t = torch.tensor(off, dtype=torch.int32, device="cuda")
    gemm(ffn, a, sa, w, sw, t, torch.bfloat16)
    gemm(ffn, *inputs(5, 12, 3, 256, 4096), t, torch.bfloat16)
    glu(ffn, a, sa, w, sw, t)


def test_a_bad_row_stays_alone(ffn):
    """NaN codes and infinite scales in one row, or in rows past an expert's end, do not reach other rows."""
    a, sa, w, sw = inputs(6, 140, 2, 256, 384, integers=True)
    off = offsets_of([70, 70])
    P, _ = ref.product(a, sa, w, sw, off.tolist())
    a.view(torch.uint8)[69, :] = 0x7F
    sa[71] = float("inf")
    out = gemm(ffn, a, sa, w, sw, off, torch.float32).double()
    keep = [i for i in range(140) if i not in (69, 71)]
    assert torch.equal(out[keep], P[keep]) and torch.isnan(out[69]).all()


def test_offsets_past_32_bits(ffn):
    """More than 2^32 bytes of rows out, and of weights."""
    rows, N = 300_001, 8192
    g = torch.Generator(device="cuda").manual_seed(7)
    a, sa = codes(g, rows, 128), scales(g, rows, 1)
    w, sw = codes(g, 1, N, 128), scales(g, 1, N // 128, 1)
    out = torch.empty(rows, N, dtype=torch.bfloat16, device="cuda")
    ffn.expert_gemm_fp8(a, sa, w, sw, out)
    P, S = ref.product(a[-200:], sa[-200:], w, sw)
    assert ((out[-200:].double() - P).abs() <= 2.0 ** -8 * P.abs() + ref.product_error(1) * S).all()
    del out
    E, N, K = 600, 2048, 4096
    w = torch.randint(0, 127, (E, N, K), dtype=torch.uint8, device="cuda", generator=g)
    sw = scales(g, E, N // 128, K // 128)
    counts = [0] * E
    counts[0], counts[E - 1] = 2, 3
    a, sa = codes(g, 5, K), scales(g, 5, K // 128)
    out = torch.empty(5, N, device="cuda")
    ffn.expert_gemm_fp8(a, sa, w, sw, out, expert_offsets=offsets_of(counts))
    w8 = w.view(torch.float8_e4m3fn)
    for rows_of, e in ((slice(0, 2), 0), (slice(2, 5), E - 1)):
        P, S = ref.product(a[rows_of], sa[rows_of], w8[e:e + 1], sw[e:e + 1])
        assert ((out[rows_of].double() - P).abs() <= ref.product_error(32) * S).all()


def test_same_result_every_time_and_on_another_stream(ffn):
    args = inputs(8, 1000, 4, 1024, 1024)
    off = offsets_of([400, 0, 500, 100])
    assert torch.equal(gemm(ffn, *args, off, torch.bfloat16), gemm(ffn, *args, off, torch.bfloat16, torch.cuda.Stream()))
    a, b = glu(ffn, *args, off), glu(ffn, *args, off, torch.cuda.Stream())
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_in_a_cuda_graph(ffn):
    a, sa, w, sw = inputs(9, 200, 2, 256, 256, integers=True)
    off, out = offsets_of([150, 50]), torch.zeros(200, 256, device="cuda")
    ffn.expert_gemm_fp8(a, sa, w, sw, out, expert_offsets=off)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ffn.expert_gemm_fp8(a, sa, w, sw, out, expert_offsets=off)
    off.copy_(offsets_of([20, 180]))
    out.zero_()
    graph.replay()
    P, _ = ref.product(a, sa, w, sw, off.tolist())
    assert torch.equal(out.double(), P)


def test_refusals(ffn):
    from combine_route_count_gb300 import moe
    a, sa, w, sw = inputs(10, 8, 2, 256, 256)
    off, out = offsets_of([4, 4]), torch.zeros(8, 256, device="cuda")
    hq, hs = torch.zeros(8, 128, dtype=torch.uint8, device="cuda"), torch.zeros(8, 1, device="cuda")
    for args, kw in [((a.float(), sa, w, sw, out), dict(expert_offsets=off)), ((a, sa, w, sw, out), {}),
                     ((a, sa[:, :1], w, sw, out), dict(expert_offsets=off)),
                     ((a, sa, w, sw[:1], out), dict(expert_offsets=off)),
                     ((a, sa, w, sw, out[:, :128]), dict(expert_offsets=off)),
                     ((a, sa, w, sw, out.half()), dict(expert_offsets=off)),
                     ((a, sa, w, sw, out), dict(expert_offsets=off[:2])),
                     ((a, sa, w, sw, out), dict(expert_offsets=off.long())),
                     ((a, sa, w, sw, out), dict(expert_offsets=off, status=off)),
                     ((a[:, :200], sa, w[:, :, :200], sw, out), dict(expert_offsets=off)),
                     ((a[:, :200].contiguous(), sa, w[:, :, :200].contiguous(), sw, out), dict(expert_offsets=off))]:
        with pytest.raises(moe.MoEError) as e:
            ffn.expert_gemm_fp8(*args, **kw)
        assert e.value.code == moe.MOE_EINVAL
    for args in [(a, sa, w, sw, hq[:4], hs), (a, sa, w, sw, hq, hs[:4]), (a, sa, w, sw, hq.int(), hs),
                 (a, sa, w[:, :128].contiguous(), sw[:, :1].contiguous(), hq, hs)]:
        with pytest.raises(moe.MoEError) as e:
            ffn.expert_glu_fp8(*args, expert_offsets=off)
        assert e.value.code == moe.MOE_EINVAL
    assert (out == 0).all() and (hq == 0).all()


def test_no_rows(ffn):
    a, sa, w, sw = inputs(11, 0, 2, 256, 256)
    ffn.expert_gemm_fp8(a, sa, w, sw, torch.empty(0, 256, device="cuda"), expert_offsets=offsets_of([0, 0]))
    ffn.expert_glu_fp8(a, sa, w, sw, torch.empty(0, 128, dtype=torch.uint8, device="cuda"),
                       torch.empty(0, 1, device="cuda"), expert_offsets=offsets_of([0, 0]))
