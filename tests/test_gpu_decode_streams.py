"""DecodeLayer on streams other than the one it was built on, without a device synchronisation between."""
import gc

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

from test_gpu_decode_layer import ffn, run, tokens, weights  # noqa: E402,F401


def occupy(ms):
    """Work on the current stream that takes about this long."""
    torch.cuda._sleep(int(ms * 2.0e6))


def test_building_stream_is_busy(ffn):  # noqa: F811
    """What the building stream has yet to do does not undo the status of a call on another stream."""
    from combine_route_count_gb300 import moe
    ws = weights(1, 8, 256, 128)
    x, sx, idx, w = tokens(2, 6, 256, 2, 8)
    run(ffn.DecodeLayer(6, 2, *ws), x, sx, idx, w)  # everything is loaded
    idx[3, 1] = 8
    out = torch.full((6, 256), -7.25, dtype=torch.bfloat16, device="cuda")
    builder, caller = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(builder):
        # The block that the status word will take is still being written.
        before = torch.empty(1, dtype=torch.int32, device="cuda")
        occupy(100)
        before.zero_()
        del before
        layer = ffn.DecodeLayer(6, 2, *ws)
    layer.forward(x, sx, idx, w, out, stream=caller)
    caller.synchronize()
    builder.synchronize()
    assert layer.get_error(caller) == moe.MOE_EROUTE
    assert (out == -7.25).all()


@pytest.mark.parametrize("T", [1, 24])
def test_layer_dropped_while_a_call_is_in_flight(ffn, T):  # noqa: F811
    """The workspace of a dropped layer is not given to others while a call on a side stream uses it."""
    ws, tk = weights(3, 16, 512, 384), tokens(4, T, 512, 4, 16)
    layer = ffn.DecodeLayer(T, 4, *ws)
    want, out = run(layer, *tk), torch.empty(T, 512, dtype=torch.bfloat16, device="cuda")
    side = torch.cuda.Stream()
    del layer
    gc.collect()
    torch.cuda.synchronize()
    layer = ffn.DecodeLayer(T, 4, *ws)
    nbytes, address = layer.workspace.numel(), layer.workspace.data_ptr()
    with torch.cuda.stream(side):
        occupy(50)
    layer.forward(*tk, out, stream=side)
    del layer
    gc.collect()
    others = [torch.empty(nbytes, dtype=torch.uint8, device="cuda") for _ in range(8)]
    assert not side.query()  # the call has not ended yet
    assert all(t.data_ptr() != address for t in others)
    side.synchronize()
    assert torch.equal(out, want)


def test_streams_as_forward_takes_them(ffn):  # noqa: F811
    from combine_route_count_gb300 import moe
    ws, tk = weights(5, 8, 256, 128), tokens(6, 6, 256, 2, 8)
    layer = ffn.DecodeLayer(6, 2, *ws)
    want, side = run(layer, *tk), torch.cuda.Stream()
    torch.cuda.synchronize()
    for stream in (None, side, side.cuda_stream, 0):
        out = torch.zeros(6, 256, dtype=torch.bfloat16, device="cuda")
        torch.cuda.synchronize()
        layer.forward(*tk, out, stream=stream)
        assert layer.get_error(stream) == moe.MOE_OK
        assert torch.equal(out, want)


def test_status_is_of_the_last_call_with_tokens(ffn):  # noqa: F811
    from combine_route_count_gb300 import moe
    layer = ffn.DecodeLayer(6, 2, *weights(7, 8, 256, 128))
    assert layer.get_error() == moe.MOE_OK
    tk = tokens(8, 6, 256, 2, 8)
    empty = [t[:0] for t in tk] + [torch.empty(0, 256, dtype=torch.bfloat16, device="cuda")]
    layer.forward(*empty)
    assert layer.get_error() == moe.MOE_OK
    tk[2][0, 0] = -1
    layer.forward(*tk, torch.empty(6, 256, dtype=torch.bfloat16, device="cuda"))
    assert layer.get_error() == moe.MOE_EROUTE
    layer.forward(*empty)
    assert layer.get_error() == moe.MOE_EROUTE


def test_built_and_called_in_a_capture(ffn):  # noqa: F811
    ws, tk = weights(9, 8, 256, 128), tokens(10, 6, 256, 2, 8)
    want, out = run(ffn.DecodeLayer(6, 2, *ws), *tk), torch.zeros(6, 256, dtype=torch.bfloat16, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer = ffn.DecodeLayer(6, 2, *ws)
        layer.forward(*tk, out)
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want) and int(layer.status) == 0
