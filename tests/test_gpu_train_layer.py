"""examples/train_expert_layer.py: router, dispatch, products, combine and all their gradients together.

The step's outputs are compared with the same layer in 64 bits, differentiated by
autograd, with the step's own choice of experts.  Between the operators lie
roundings to bf16, half a step (2^-8) each; the norms of a result's error are
bounded by as many of them as lie on its way, added up, with a factor of 2 for
what the products and activations between make of them (their norms on these
random weights: a product with normalised weights 1, |SiLU'| < 1.1)."""
import importlib.util
import os

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from combine_route_count_gb300 import build, moe
    build.build()
    build.build_train()
    moe.load_library()
    spec = importlib.util.spec_from_file_location("train_expert_layer", os.path.join(ROOT, "examples", "train_expert_layer.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def swiglu(v):
    n = v.shape[1] // 2
    return v[:, :n] * torch.sigmoid(v[:, :n]) * v[:, n:]


def reference(layer, x, d_out):
    W = {k: v.double().requires_grad_() for k, v in layer.weights.items()}
    x = x.double().requires_grad_()
    logits = x @ W["router"].t()
    logits.retain_grad()
    idx = layer.idx.long()
    p = torch.sigmoid(logits).gather(1, idx)
    w = p / p.sum(1, keepdim=True)
    w.retain_grad()
    out = swiglu(x @ W["s13"].t()) @ W["s2"].t()
    for e in range(layer.E):
        t, k = (idx == e).nonzero(as_tuple=True)
        if len(t):
            y = swiglu(x[t] @ W["w13"][e].t()) @ W["w2"][e].t()
            out = out.index_add(0, t, w[t, k][:, None] * y)
    out.backward(d_out.double())
    return out.detach(), x.grad, w.grad, logits.grad, {k: v.grad for k, v in W.items()}


def near(name, got, want, roundings):
    far = float((got.double() - want).norm() / want.norm())
    assert far <= 2 * roundings * 2.0 ** -8, (name, far)


@pytest.mark.parametrize("tokens,hidden,inter,shared,experts,top_k", [
    (300, 512, 256, 128, 16, 4), (64, 256, 128, 256, 8, 2), (1, 512, 64, 64, 8, 4), (1000, 1032, 72, 200, 40, 6)])
def test_step(example, tokens, hidden, inter, shared, experts, top_k):
    layer, x, d_out, out, (dx, dw, d_logits, grads) = example.run(tokens, hidden, inter, shared, experts, top_k)
    want, want_x, want_w, want_l, want_g = reference(layer, x, d_out)
    near("out", out, want, 5)                   # logits, h, expert_y, combined, out
    near("x", dx, want_x, 8)                    # pre, h of the slopes; d_y, d_pre, d_ex, dx twice, the sum
    near("w", dw, want_w, 4)                    # h, expert_y; the logits
    # The router's gradient is a difference of the weights' gradients: its errors are theirs.
    scale = float((layer.w.double() * want_w).norm())
    assert float((d_logits.double() - want_l).norm()) <= 2 * 5 * 2.0 ** -8 * scale
    near("w2", grads["w2"], want_g["w2"], 3)    # h, w, d_y
    near("w13", grads["w13"], want_g["w13"], 5)  # d_y, pre, d_pre, w
    near("s2", grads["s2"], want_g["s2"], 2)
    near("s13", grads["s13"], want_g["s13"], 4)
    far = float((grads["router"].double() - want_g["router"]).norm())
    assert far <= 2 * 6 * 2.0 ** -8 * scale * float(x.double().norm(dim=1).max())


def test_step_in_a_graph_and_again(example):
    """The same bits in a captured step, and for other tokens in a replay of it."""
    layer, x, d_out, out, (dx, dw, d_logits, grads) = example.run(200, 512, 128, 64, 8, 2)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out2 = layer.forward(x)
        dx2, dw2, dl2, grads2 = layer.backward(d_out)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, out2) and torch.equal(dx, dx2) and torch.equal(dw, dw2) and torch.equal(d_logits, dl2)
    assert all(torch.equal(grads[k], grads2[k]) for k in grads)
    x.copy_(torch.randn_like(x))
    graph.replay()
    torch.cuda.synchronize()
    got = [t.clone() for t in (out2, dx2, dw2, dl2, *grads2.values())]
    eager = layer.forward(x)
    dx3, dw3, dl3, grads3 = layer.backward(d_out)
    assert all(torch.equal(a, b) for a, b in zip(got, (eager, dx3, dw3, dl3, *grads3.values())))
    layer.check()


def test_steps_on_two_streams_at_once(example):
    """Two layers' steps side by side: nothing is shared between calls."""
    sizes = [(300, 512, 256, 128, 16, 4), (257, 264, 72, 200, 40, 6)]
    alone = [example.run(*s, seed=i) for i, s in enumerate(sizes)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sizes]
    results = [[], []]
    for _ in range(5):
        for (layer, x, d_out, _, _), s, r in zip(alone, streams, results):
            with torch.cuda.stream(s):
                out = layer.forward(x)
                dx, dw, dl, grads = layer.backward(d_out)
                r.append((out, dx, dw, dl, *grads.values()))
    torch.cuda.synchronize()
    for (_, _, _, out, (dx, dw, dl, grads)), r in zip(alone, results):
        for again in r:
            assert all(torch.equal(a, b) for a, b in zip((out, dx, dw, dl, *grads.values()), again))
