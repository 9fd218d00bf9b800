"""Argument checks of the training operators that run before any CUDA call,
through the C ABI.  No GPU is needed."""
import pytest


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


A, BAD = 0x1000, 0x1008  # addresses that are never read: every call below is refused on the host


def test_router_checks(moe):
    def forward(z=A, t=1, b=None, T=4, E=8, K=2, s=0, scale=1.0, i=A, w=A):
        return refused(moe, moe.moe_router_topk, z, t, b, T, E, K, s, True, scale, i, w)

    def backward(z=A, t=1, i=A, dw=A, T=4, E=8, K=2, s=0, scale=1.0, d=A):
        return refused(moe, moe.moe_router_topk_backward, z, t, i, dw, T, E, K, s, True, scale, d)

    for kw in (dict(z=None), dict(t=2), dict(t=-1), dict(T=-1), dict(T=2 ** 31), dict(E=0), dict(E=1025), dict(K=0),
               dict(K=9), dict(K=17, E=32), dict(s=2), dict(s=-1), dict(scale=float("inf")), dict(scale=float("nan")),
               dict(i=None), dict(z=0x1002), dict(z=0x1001, t=0), dict(i=0x1002)):
        assert forward(**kw) and backward(**kw), kw
    assert forward(w=None) and forward(b=A) and forward(b=0x1002, s=1) and forward(w=0x1002)
    assert backward(dw=None) and backward(d=None) and backward(dw=0x1002) and backward(d=0x1002)
    moe.moe_router_topk(None, 1, None, 0, 8, 2, 0, True, 1.0, None, None, stream=0)  # no tokens: nothing to do
    moe.moe_router_topk_backward(None, 1, None, None, 0, 8, 2, 0, True, 1.0, None, stream=0)


def test_move_checks(moe):
    def combine(g=A, y=A, w=A, s=A, T=4, H=64, K=2, rows=8, dy=A, dw=A):
        return refused(moe, moe.moe_combine_backward, g, y, w, s, T, H, K, rows, dy, dw)

    def dispatch(d=A, s=A, add=None, T=4, H=64, K=2, rows=8, x=A):
        return refused(moe, moe.moe_dispatch_backward, d, s, add, T, H, K, rows, x)

    for kw in (dict(s=None), dict(s=0x1002), dict(T=-1), dict(T=2 ** 31), dict(T=2 ** 30, K=2), dict(H=0), dict(H=60),
               dict(H=-8), dict(K=0), dict(K=17), dict(rows=-1), dict(rows=2 ** 31)):
        assert combine(**kw) and dispatch(**kw), kw
    for kw in (dict(g=None), dict(w=None), dict(dy=None), dict(y=None), dict(dw=None), dict(g=BAD), dict(y=BAD),
               dict(dy=BAD), dict(w=0x1002), dict(dw=0x1002)):
        assert combine(**kw), kw
    for kw in (dict(d=None), dict(x=None), dict(d=BAD), dict(x=BAD), dict(add=BAD)):
        assert dispatch(**kw), kw
    moe.moe_combine_backward(None, None, None, None, 0, 64, 2, 8, None, None, stream=0)
    moe.moe_dispatch_backward(None, None, None, 0, 64, 2, 8, None, stream=0)


def test_product_checks(moe):
    def forward(a=A, rows=4, k=64, w=A, n=64, E=2, off=A, b=A, bt=1, act=0, r=A, pre=A, out=A, t=0, st=None):
        return refused(moe, moe.moe_expert_linear, a, rows, k, w, n, E, off, b, bt, act, r, pre, out, t, st)

    def by_rows(a=A, rows=4, k=64, w=A, n=64, E=2, off=A, act=1, pre=A, out=A, st=None):
        return refused(moe, moe.moe_expert_linear_backward_input, a, rows, n, w, k, E, off, act, pre, out, st)

    def by_weights(a=A, rows=4, k=64, w=A, n=64, E=2, off=A, out=A, t=0, b=A, st=None):
        return refused(moe, moe.moe_expert_linear_backward_weight, a, rows, n, w, k, E, off, out, t, b, False, st)

    for kw in (dict(a=None), dict(w=None), dict(out=None), dict(a=BAD), dict(w=BAD), dict(out=BAD), dict(off=0x1002),
               dict(st=0x1002), dict(rows=-1), dict(rows=2 ** 31 - 1), dict(k=0), dict(k=-8), dict(k=60), dict(n=0),
               dict(n=60), dict(n=2 ** 30 + 8), dict(k=2 ** 30 + 8), dict(E=0), dict(E=1025), dict(off=None)):
        assert forward(**kw) and by_rows(**kw) and by_weights(**kw), kw
    for kw in (dict(b=BAD), dict(bt=2), dict(act=-1), dict(act=5), dict(act=4, n=72), dict(r=BAD), dict(pre=BAD),
               dict(t=2), dict(r=A, out=A, t=1)):
        assert forward(**kw), kw
    for kw in (dict(act=0), dict(pre=None), dict(act=-1), dict(act=5), dict(pre=BAD)):
        assert by_rows(**kw), kw
    for kw in (dict(t=2), dict(b=BAD)):
        assert by_weights(**kw), kw
    moe.moe_expert_linear(None, 0, 64, None, 64, 2, A, None, 0, 0, None, None, None, 0, stream=0)
    moe.moe_expert_linear_backward_input(None, 0, 64, None, 64, 2, A, 0, None, None, stream=0)
    moe.moe_expert_linear_backward_weight(None, 0, 64, None, 64, 2, A, A, 0, None, True, stream=0)


def test_names(moe):
    pytest.importorskip("torch")
    from combine_route_count_gb300 import train
    for call in (lambda: train.router_topk(None, None, None, score="tanh"),
                 lambda: train.expert_linear(None, None, None, activation=["silu"])):
        try:
            call()
        except moe.MoEError as e:
            assert e.code == moe.MOE_EINVAL and "must be one of" in str(e)
        else:
            raise AssertionError("not refused")
