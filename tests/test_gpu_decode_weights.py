"""DecodeLayer reads the weights where its tensors have them at the call."""
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

from test_gpu_decode_layer import ffn, run, tokens, weights  # noqa: E402,F401


def put(t, other, how):
    if how == "data":
        t.data = other
    elif how == "set_":
        t.set_(other)
    else:
        t.copy_(other)


@pytest.mark.parametrize("how", ["data", "set_", "copy_"])
@pytest.mark.parametrize("which", [0, 1, 2, 3])
def test_replaced_weights(ffn, how, which):  # noqa: F811
    ws, new, tk = list(weights(1, 8, 256, 128)), weights(2, 8, 256, 128), tokens(3, 6, 256, 2, 8)
    layer = ffn.DecodeLayer(6, 2, *ws)
    old = run(layer, *tk)
    storages = [w.untyped_storage() for w in ws]  # the old memory stays valid
    want = run(ffn.DecodeLayer(6, 2, *[new[i] if i == which else ws[i] for i in range(4)]), *tk)
    assert not torch.equal(old, want)
    put(ws[which], new[which], how)
    assert torch.equal(run(layer, *tk), want)
    del storages


def test_weights_that_no_longer_fit_are_refused(ffn):  # noqa: F811
    from combine_route_count_gb300 import moe
    tk, out = tokens(3, 6, 256, 2, 8), torch.zeros(6, 256, dtype=torch.bfloat16, device="cuda")
    for other in (lambda w: w.cpu(), lambda w: w[:, :128].contiguous(), lambda w: w.half(), lambda w: w[:4].clone()):
        for which in range(4):
            ws = list(weights(1, 8, 256, 128))
            storages = [w.untyped_storage() for w in ws]
            layer = ffn.DecodeLayer(6, 2, *ws)
            new = other(ws[which])
            if new.shape == ws[which].shape and new.dtype == ws[which].dtype and new.device == ws[which].device:
                continue  # the cut leaves a tensor of scales as it is
            if new.device == ws[which].device and new.dtype == ws[which].dtype:
                ws[which].data = new
            else:
                layer._weights = tuple(new if i == which else ws[i] for i in range(4))
            with pytest.raises(moe.MoEError) as e:
                layer.forward(*tk, out)
            assert e.value.code == moe.MOE_EINVAL
            del storages
    assert (out == 0).all()
