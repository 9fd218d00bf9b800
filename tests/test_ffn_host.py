"""Argument checks of the feed-forward operators that run before any CUDA
call, through the C ABI; and the tests' own 64-bit forms.  No GPU is needed."""
import numpy as np
import pytest

import ffn_ref as ref


@pytest.fixture(scope="module")
def moe():
    from combine_route_count_gb300 import build, moe as m
    build.build()
    m.load_library()
    return m


def refused(moe, fn, *args):
    with pytest.raises(moe.MoEError) as e:
        fn(*args, stream=0)
    return e.value.code == moe.MOE_EINVAL


def test_e4m3_grid():
    torch = pytest.importorskip("torch")
    codes = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).float().numpy().astype(np.float64)
    codes = codes[np.isfinite(codes)]
    assert np.array_equal(ref.e4m3(codes), codes)
    v = np.random.default_rng(0).standard_normal(20000) * 10.0 ** np.random.default_rng(1).uniform(-4, 2.6, 20000)
    want = torch.from_numpy(np.clip(v, -448, 448)).to(torch.float8_e4m3fn).float().numpy()
    assert np.array_equal(ref.e4m3(v), want)


def test_add_rms_norm_checks(moe):
    A, bad = 0x1000, 0x1008  # addresses that are never read: every call below is refused on the host

    def call(x=A, r=None, w=A, wt=0, T=4, H=256, eps=1e-6, ro=None, y=None, q=A, s=A):
        return refused(moe, moe.moe_add_rms_norm_fp8, x, r, w, wt, T, H, eps, ro, y, q, s)

    for kw in (dict(x=None), dict(w=None), dict(q=None), dict(s=None), dict(x=bad), dict(w=bad), dict(q=bad),
               dict(y=bad), dict(s=0x1002), dict(r=A), dict(ro=A), dict(r=bad, ro=A), dict(r=A, ro=bad), dict(wt=2),
               dict(T=-1), dict(T=2 ** 31), dict(H=0), dict(H=200), dict(H=65536 + 128), dict(eps=-1.0), dict(eps=0.0),
               dict(eps=float("inf")), dict(eps=float("nan")), dict(r=A, ro=A, y=A)):
        assert call(**kw), kw
    moe.moe_add_rms_norm_fp8(None, None, None, 0, 0, 256, 1e-6, None, None, None, None, stream=0)  # no tokens: nothing to do


def test_product_checks(moe):
    A, bad = 0x1000, 0x1008

    def gemm(a=A, s=A, rows=4, k=256, w=A, ws=A, n=256, E=2, off=A, out=A, t=0, st=None):
        return refused(moe, moe.moe_expert_gemm_fp8, a, s, rows, k, w, ws, n, E, off, out, t, st)

    def glu(a=A, s=A, rows=4, k=256, w=A, ws=A, n=256, E=2, off=A, out=A, hs=A, st=None):
        return refused(moe, moe.moe_expert_glu_fp8, a, s, rows, k, w, ws, n, E, off, out, hs, st)

    for kw in (dict(a=None), dict(s=None), dict(w=None), dict(ws=None), dict(out=None), dict(a=bad), dict(w=bad),
               dict(out=bad), dict(s=0x1002), dict(ws=0x1002), dict(off=0x1002), dict(st=0x1002), dict(rows=-1),
               dict(rows=2 ** 31 - 1), dict(k=0), dict(k=-16), dict(k=200), dict(n=0), dict(E=0), dict(E=1025),
               dict(off=None), dict(n=2 ** 30)):
        assert gemm(**kw) and glu(**kw), kw
    assert gemm(t=2) and gemm(n=260) and glu(n=192) and glu(hs=None) and glu(hs=0x1002)
    moe.moe_expert_gemm_fp8(None, None, 0, 256, None, None, 256, 2, A, None, 0, None, stream=0)


def test_decode_layer_checks(moe):
    A, bad = 0x1000, 0x1008

    def call(T=4, H=256, K=2, E=8, N=1, I=128, x=A, sx=A, idx=A, w=A, a=A, sa=A, b=A, sb=A, out=A, st=A, ws=A, n=1 << 20):
        return refused(moe, moe.moe_decode_layer_fp8, moe.make_config(T, H, K, E, N), I, x, sx, idx, w, a, sa, b, sb,
                       out, st, ws, n)

    for kw in (dict(T=65), dict(T=-1), dict(H=200), dict(H=0), dict(K=0), dict(K=9), dict(K=17, E=32), dict(E=1032),
               dict(N=3), dict(I=0), dict(I=64), dict(I=-128), dict(x=None), dict(sx=None), dict(idx=None),
               dict(w=None), dict(a=None), dict(sa=None), dict(b=None), dict(sb=None), dict(out=None), dict(st=None),
               dict(ws=None), dict(x=bad), dict(a=bad), dict(b=bad), dict(out=bad), dict(ws=0x1010), dict(n=1024),
               dict(idx=0x1002), dict(w=0x1002), dict(sx=0x1002), dict(st=0x1002)):
        assert call(**kw), kw
    assert moe.moe_decode_workspace_bytes(moe.make_config(4, 256, 2, 8, 1), 128) == 8 * 128 + 256
    with pytest.raises(moe.MoEError):
        moe.moe_decode_workspace_bytes(moe.make_config(65, 256, 2, 8, 1), 128)
    moe.moe_decode_layer_fp8(moe.make_config(0, 256, 2, 8, 1), 128, *[None] * 11, 0, stream=0)
