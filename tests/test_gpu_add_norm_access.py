"""The forms of moe_add_rms_norm_fp8's loads and stores: a call's rows are those that the same rows give in small
calls (which test_gpu_add_norm.py compares with the formula), bit for bit, whatever the call's size makes it take."""
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

from test_gpu_add_norm import ffn  # noqa: E402,F401


def call(ffn, x, w, r, want_y):  # noqa: F811
    T, H = x.shape
    q, s = torch.empty(T, H, dtype=torch.uint8, device="cuda"), torch.empty(T, H // 128, device="cuda")
    ro, y = None if r is None else torch.empty_like(x), torch.empty_like(x) if want_y else None
    ffn.add_rms_norm_fp8(x, w, q, s, residual=r, residual_out=ro, y=y)
    return [t for t in (q, s, ro, y) if t is not None]


# More than 2^25 and 2^26 elements, from short rows to those that are walked twice.
@pytest.mark.parametrize("T,H", [(32773, 1024), (65539, 1024), (4700, 7168), (9400, 7168), (8193, 8192), (5500, 12288),
                                 (2051, 16384), (1027, 32768), (2049, 32768)])
@pytest.mark.parametrize("residual", [True, False])
@pytest.mark.parametrize("want_y", [True, False])
@pytest.mark.parametrize("f32", [True, False])
def test_rows_of_a_large_call(ffn, T, H, residual, want_y, f32):  # noqa: F811
    g = torch.Generator(device="cuda").manual_seed(T + H)
    x = torch.randn(T, H, generator=g, device="cuda").to(torch.bfloat16)
    r = torch.randn(T, H, generator=g, device="cuda").to(torch.bfloat16) if residual else None
    w = torch.randn(H, generator=g, device="cuda")
    w = w if f32 else w.to(torch.bfloat16)
    out = call(ffn, x, w, r, want_y)
    for lo in range(0, T, 500):
        part = call(ffn, x[lo:lo + 500], w, None if r is None else r[lo:lo + 500], want_y)
        assert all(torch.equal(a[lo:lo + 500], b) for a, b in zip(out, part)), lo
