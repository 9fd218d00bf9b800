"""moe_add_rms_norm_fp8 on the GPU against the formula in 64 bits.

Tolerances: the kernel works in float32.  A row's sum of squares adds at most
H <= 65536 positive terms, in chains of at most 16 * H / 16384 per thread, a
five-step tree and at most 32 partial sums: its relative error is below
(16 * 4 + 5 + 32 + 2) * 2^-24 < 7e-6, halved by the square root; the products
add 3 * 2^-24 and the reciprocal root 2^-22.  So every v is within 4e-6 of its
own size: REL.  residual_out has one right value, the float32 sum rounded to
bf16, and is compared bit for bit; y is that far from v plus one rounding,
half a bf16 step of v's binade."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

import ffn_ref as ref  # noqa: E402

REL = 4e-6


def bf16_half_step(v):
    _, e = np.frexp(np.abs(v))  # |v| < 2^e, eight significant bits
    return np.exp2(e - 9.0)


@pytest.fixture(scope="module")
def ffn():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from combine_route_count_gb300 import build, ffn as f, moe
    build.build()
    build.build_ffn()
    moe.load_library()
    return f


def run(ffn, x, weight, residual=None, want_y=True, eps=1e-6, inplace=False, stream=None):
    T, H = x.shape
    guard = 1
    q = torch.full((T + 2 * guard, H), 0x5A, dtype=torch.uint8, device="cuda")
    s = torch.full((T + 2 * guard, H // 128), -7.25, device="cuda")
    xd, wd = x.cuda(), weight.cuda()
    rd = residual.cuda() if residual is not None else None
    ro = None if rd is None else (rd if inplace else torch.empty_like(rd))
    y = (xd if inplace else torch.empty_like(xd)) if want_y else None
    torch.cuda.synchronize()
    ffn.add_rms_norm_fp8(xd, wd, q[guard:guard + T], s[guard:guard + T], eps=eps, residual=rd, residual_out=ro, y=y,
                         stream=stream)
    torch.cuda.synchronize()
    for edge in (slice(0, guard), slice(guard + T, None)):
        assert (q[edge] == 0x5A).all() and (s[edge] == -7.25).all()
    codes = q[guard:guard + T].view(torch.float8_e4m3fn).float()
    return ref.f64(codes), ref.f64(s[guard:guard + T]), ro, y


def check(ffn, x, weight, residual=None, want_y=True, eps=1e-6, inplace=False):
    q, scales, ro, y = run(ffn, x, weight, residual, want_y, eps, inplace)
    s64, v64 = ref.add_norm(ref.f64(x), None if residual is None else ref.f64(residual), ref.f64(weight), eps)
    ref.assert_codes_near(q, scales, v64, REL)
    if residual is not None:
        assert torch.equal(ro.cpu(), (x.float() + residual.float()).to(torch.bfloat16))
    if want_y:
        assert np.all(np.abs(ref.f64(y) - v64) <= bf16_half_step(v64 * (1 + REL)) + REL * np.abs(v64))


@pytest.mark.parametrize("T", [1, 2, 7, 64, 1000])
@pytest.mark.parametrize("H", [128, 256, 512, 640, 4096, 7168, 16384])
def test_sizes(ffn, T, H):
    rng = np.random.default_rng(T * 1000 + H)
    x, r = ref.bf16(rng, T, H), ref.bf16(rng, T, H, scale=3.0)
    check(ffn, x, 1.0 + ref.bf16(rng, H, scale=0.2), r)


@pytest.mark.parametrize("H", [16512, 32768, 65536])
@pytest.mark.parametrize("residual", [True, False])
def test_long_rows(ffn, H, residual):
    rng = np.random.default_rng(H)
    x = ref.bf16(rng, 5, H)
    check(ffn, x, ref.bf16(rng, H), ref.bf16(rng, 5, H) if residual else None, inplace=True)


@pytest.mark.parametrize("residual", [True, False])
@pytest.mark.parametrize("want_y", [True, False])
@pytest.mark.parametrize("f32", [True, False])
@pytest.mark.parametrize("inplace", [True, False])
def test_forms(ffn, residual, want_y, f32, inplace):
    rng = np.random.default_rng(5)
    x = ref.bf16(rng, 333, 1152)
    w = ref.bf16(rng, 1152)
    if f32:
        w = torch.from_numpy(rng.standard_normal(1152).astype(np.float32))
    check(ffn, x, w, ref.bf16(rng, 333, 1152) if residual else None, want_y, inplace=inplace)


def test_many_more_rows_than_ctas(ffn):
    rng = np.random.default_rng(6)
    check(ffn, ref.bf16(rng, 9001, 256), ref.bf16(rng, 256), ref.bf16(rng, 9001, 256))


@pytest.mark.parametrize("H", [640, 20480])
@pytest.mark.parametrize("residual", [True, False])
def test_rows_on_16_byte_boundaries(ffn, H, residual):
    """Rows that begin between 32-byte sectors take other loads and stores; the results are the same bits."""
    T, rng = 37, np.random.default_rng(H)
    x, r, w = ref.bf16(rng, T, H), ref.bf16(rng, T, H), ref.bf16(rng, H)
    q0, s0, ro0, y0 = run(ffn, x, w, r if residual else None)

    def shifted(t):  # a copy 16 bytes past a sector's beginning
        buf = torch.empty(T * H + 16, dtype=torch.bfloat16, device="cuda")
        v = buf[8:8 + T * H].view(T, H)
        assert v.data_ptr() % 32 == 16
        return v.copy_(t)

    xd, rd = shifted(x), shifted(r) if residual else None
    y, ro = shifted(torch.zeros_like(x)), shifted(torch.zeros_like(x)) if residual else None
    q = torch.empty(T, H, dtype=torch.float8_e4m3fn, device="cuda")
    s = torch.empty(T, H // 128, device="cuda")
    ffn.add_rms_norm_fp8(xd, w.cuda(), q, s, residual=rd, residual_out=ro, y=y)
    assert np.array_equal(ref.f64(q.float()), q0) and np.array_equal(ref.f64(s), s0)
    assert torch.equal(y, y0) and (not residual or torch.equal(ro, ro0))


def test_offsets_past_32_bits(ffn):
    """More than 2^32 bytes of x and more than 2^31 codes: the last rows are right."""
    T, H = 131072 + 3, 16384
    rng = np.random.default_rng(7)
    x = torch.zeros(T, H, dtype=torch.bfloat16, device="cuda")
    tail = ref.bf16(rng, 3, H)
    x[-3:] = tail.cuda()
    w = ref.bf16(rng, H)
    q = torch.empty(T, H, dtype=torch.float8_e4m3fn, device="cuda")
    s = torch.empty(T, H // 128, device="cuda")
    ffn.add_rms_norm_fp8(x, w.cuda(), q, s)
    _, v = ref.add_norm(ref.f64(tail), None, ref.f64(w), 1e-6)
    ref.assert_codes_near(ref.f64(q[-3:].float()), ref.f64(s[-3:]), v, REL)
    assert (q[:4].float() == 0).all() and (s[:4] == 1).all()


def test_special_rows(ffn):
    """All-zero rows and blocks, tiny and huge values; a NaN or an infinity stays in its row."""
    rng = np.random.default_rng(8)
    x = ref.bf16(rng, 8, 512)
    w = torch.ones(512)
    x[1] = 0
    x[2, 128:256] = 0
    x[3] *= 2.0 ** -80   # the norm's eps dominates: v far below the floor of the scales
    x[4] *= 2.0 ** 50
    x[5, 17] = float("nan")
    x[6, 300] = float("inf")
    q, s, _, y = run(ffn, x, w)
    good = [0, 1, 2, 3, 4, 7]
    _, v = ref.add_norm(ref.f64(x)[good], None, ref.f64(w), 1e-6)
    ref.assert_codes_near(q[good], s[good], v, REL)
    assert np.all(q[1] == 0) and np.all(s[1] == 1) and s[2, 1] == 1 and np.all(q[2, 128:256] == 0)
    assert np.isfinite(q[good]).all()
    # below the floor: weights that push a block under 2^-100
    q, s, _, y = run(ffn, x[:1], torch.full((512,), 2.0 ** -110))
    assert np.allclose(s, 2.0 ** -100 / 448, rtol=1e-6) and np.isfinite(q).all() and np.abs(q).max() <= 448 * 2.0 ** -7


def test_same_result_every_time_and_on_another_stream(ffn):
    rng = np.random.default_rng(9)
    x, r, w = ref.bf16(rng, 513, 7168), ref.bf16(rng, 513, 7168), ref.bf16(rng, 7168)
    a = run(ffn, x, w, r)
    b = run(ffn, x, w, r, stream=torch.cuda.Stream())
    assert np.array_equal(a[0], b[0]) and np.array_equal(a[1], b[1])
    assert torch.equal(a[2], b[2]) and torch.equal(a[3], b[3])


def test_feeds_the_quantised_dispatch(ffn):
    """The codes of bf16 rows whose norm is exact equal those that the fp8 dispatch makes of y."""
    from combine_route_count_gb300 import moe
    T, H, E, K = 16, 512, 8, 2
    rng = np.random.default_rng(10)
    # +-1 rows: mean square 1; eps so small that 1 + eps rounds to 1
    x = torch.from_numpy(rng.choice([-1.0, 1.0], (T, H)).astype(np.float32)).to(torch.bfloat16).cuda()
    w = torch.from_numpy((2.0 ** rng.integers(-3, 4, H)).astype(np.float32)).cuda()
    q = torch.empty(T, H, dtype=torch.uint8, device="cuda")
    s, y = torch.empty(T, H // 128, device="cuda"), torch.empty_like(x)
    ffn.add_rms_norm_fp8(x, w, q, s, eps=1e-30, y=y)
    idx = torch.from_numpy(np.stack([rng.permutation(E)[:K] for _ in range(T)]).astype(np.int32)).cuda()
    eq, es = torch.empty(T * K, H, dtype=torch.uint8, device="cuda"), torch.empty(T * K, H // 128, device="cuda")
    eq2, es2 = torch.empty_like(eq), torch.empty_like(es)
    for send, args in (("dispatch_send_quantized", (q, s, idx, eq, es)), ("dispatch_send_fp8", (y, idx, eq2, es2))):
        layer = moe.MoELayer(T, H, K, E, 1)
        getattr(layer, send)(*args)
        assert layer.get_error() == moe.MOE_OK
    assert torch.equal(eq, eq2) and torch.equal(es, es2)


def test_empty(ffn):
    x = torch.empty(0, 256, dtype=torch.bfloat16, device="cuda")
    ffn.add_rms_norm_fp8(x, torch.ones(256, device="cuda"), torch.empty(0, 256, dtype=torch.uint8, device="cuda"),
                         torch.empty(0, 2, device="cuda"))


def test_refusals(ffn):
    from combine_route_count_gb300 import moe
    x = torch.zeros(4, 256, dtype=torch.bfloat16, device="cuda")
    w, q = torch.ones(256, device="cuda"), torch.zeros(4, 256, dtype=torch.uint8, device="cuda")
    s = torch.zeros(4, 2, device="cuda")
    for args, kw in [((x.float(), w, q, s), {}), ((x.cpu(), w, q, s), {}), ((x[:, ::2], w, q, s), {}),
                     ((x, w[:128], q, s), {}), ((x, w, q[:2], s), {}), ((x, w, q, s[:, :1]), {}),
                     ((x, w.half(), q, s), {}), ((x, w, q, s), dict(residual=x)), ((x, w, q, s), dict(eps=0.0)),
                     ((x, w, q, s), dict(eps=float("nan"))),
                     ((x, w, q, s), dict(residual=x, residual_out=x, y=x)),
                     ((x[:, :250].contiguous(), w[:250].contiguous(), q[:, :250].contiguous(), s[:, :1].contiguous()), {})]:
        with pytest.raises(moe.MoEError) as e:
            ffn.add_rms_norm_fp8(*args, **kw)
        assert e.value.code == moe.MOE_EINVAL
    assert (q == 0).all() and (s == 0).all()
