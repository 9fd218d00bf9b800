"""examples/fp8_expert_layer.py: norm, dispatch, both products and combine together, against the whole-layer call."""
import importlib.util
import os

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("tokens,few,hidden,inter,experts,top_k", [
    (300, 40, 1024, 256, 16, 4), (64, 64, 512, 128, 8, 2), (2000, 1, 2048, 640, 40, 6)])
def test_both_ways_agree(tokens, few, hidden, inter, experts, top_k):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from combine_route_count_gb300 import build, moe
    build.build()
    build.build_ffn()
    moe.load_library()
    spec = importlib.util.spec_from_file_location("fp8_expert_layer", os.path.join(ROOT, "examples", "fp8_expert_layer.py"))
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    many, part = example.run(tokens, few, hidden, inter, experts, top_k)
    assert torch.isfinite(many.float()).all()
    # Same codes in; what differs is expert_y's rounding to bf16 (2^-9 of each
    # of top_k terms, adding like noise) and the two outputs' own (2^-9 each).
    far = (many[:few].float() - part.float()).norm() / part.float().norm()
    assert far < 4 * 2.0 ** -9, float(far)
