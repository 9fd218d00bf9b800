"""A training step of one bf16 expert layer on one GPU: forward and every gradient.

Router (product, choice, weights), dispatch, the experts' gate/up and down
products with SwiGLU, the weighted combine, and a shared expert whose second
product adds the combined rows as its residual; then the way back through all of
it.  Tokens and weights are random.

    python examples/train_expert_layer.py [--tokens 4096]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from combine_route_count_gb300 import moe, train  # noqa: E402

BF16 = dict(dtype=torch.bfloat16, device="cuda")


class ExpertLayer:
    """Weights of one layer (experts a multiple of 8) and what the way back needs of the last forward pass."""

    def __init__(self, tokens, hidden, inter, shared, experts, top_k, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        w = lambda *s: torch.randn(*s, generator=g, **BF16) * s[-1] ** -0.5  # noqa: E731
        self.T, self.H, self.I, self.S, self.E, self.K = tokens, hidden, inter, shared, experts, top_k
        self.weights = {"router": w(experts, hidden), "w13": w(experts, 2 * inter, hidden),
                        "w2": w(experts, hidden, inter), "s13": w(2 * shared, hidden), "s2": w(hidden, shared)}
        self.bias = 0.02 * torch.randn(experts, generator=g, device="cuda")  # of the choice, kept by load balancing
        self.moe = moe.MoELayer(tokens, hidden, top_k, experts, 1)
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")

    def forward(self, x):
        W, T, rows = self.weights, self.T, self.T * self.K
        self.x, self.logits = x, torch.empty(T, self.E, **BF16)
        train.expert_linear(x, W["router"], self.logits, status=self.status)
        self.idx = torch.empty(T, self.K, dtype=torch.int32, device="cuda")
        self.w = torch.empty(T, self.K, device="cuda")
        train.router_topk(self.logits, self.idx, self.w, score="sigmoid", bias=self.bias)
        self.expert_x = torch.empty(rows, self.H, **BF16)
        self.moe.dispatch_send(x, self.idx, self.expert_x)
        self.layout = self.moe.dispatch_recv()
        off = self.layout["expert_offsets"]
        self.pre, self.h = torch.empty(rows, 2 * self.I, **BF16), torch.empty(rows, self.I, **BF16)
        train.expert_linear(self.expert_x, W["w13"], self.h, activation="swiglu", pre=self.pre, expert_offsets=off,
                            status=self.status)
        self.expert_y = torch.empty(rows, self.H, **BF16)
        train.expert_linear(self.h, W["w2"], self.expert_y, expert_offsets=off, status=self.status)
        out = torch.empty(T, self.H, **BF16)
        self.moe.combine_send(self.expert_y)
        self.moe.combine_recv(self.w, out)
        self.shared_pre, self.shared_h = torch.empty(T, 2 * self.S, **BF16), torch.empty(T, self.S, **BF16)
        train.expert_linear(x, W["s13"], self.shared_h, activation="swiglu", pre=self.shared_pre, status=self.status)
        train.expert_linear(self.shared_h, W["s2"], out, residual=out, status=self.status)
        return out

    def backward(self, d_out):
        """Gradients by x, the router's logits and every weight (float32, as an optimizer sums them)."""
        W, T, rows = self.weights, self.T, self.T * self.K
        off, slot_row, st = self.layout["expert_offsets"], self.layout["slot_row"], self.status
        grads = {k: torch.empty(v.shape, device="cuda") for k, v in W.items()}
        # the shared expert
        d_pre, dx = torch.empty(T, 2 * self.S, **BF16), torch.empty(T, self.H, **BF16)
        train.expert_linear_backward_weight(d_out, self.shared_h, grads["s2"], status=st)
        train.expert_linear_backward_input(d_out, W["s2"], d_pre, activation="swiglu", pre=self.shared_pre, status=st)
        train.expert_linear_backward_weight(d_pre, self.x, grads["s13"], status=st)
        train.expert_linear_backward_input(d_pre, W["s13"], dx, status=st)
        # the experts
        d_w = torch.empty(T, self.K, device="cuda")
        d_y = torch.empty_like(self.expert_y)
        train.combine_backward(d_out, slot_row, self.w, d_y, expert_y=self.expert_y, d_topk_w=d_w)
        train.expert_linear_backward_weight(d_y, self.h, grads["w2"], expert_offsets=off, status=st)
        d_pre = torch.empty(rows, 2 * self.I, **BF16)
        train.expert_linear_backward_input(d_y, W["w2"], d_pre, activation="swiglu", pre=self.pre, expert_offsets=off,
                                           status=st)
        train.expert_linear_backward_weight(d_pre, self.expert_x, grads["w13"], expert_offsets=off, status=st)
        d_ex = torch.empty_like(self.expert_x)
        train.expert_linear_backward_input(d_pre, W["w13"], d_ex, expert_offsets=off, status=st)
        train.dispatch_backward(d_ex, slot_row, dx, add=dx)
        # the router
        d_logits, dx_router = torch.empty_like(self.logits), torch.empty(T, self.H, **BF16)
        train.router_topk_backward(self.logits, self.idx, d_w, d_logits, score="sigmoid")
        train.expert_linear_backward_weight(d_logits, self.x, grads["router"], status=st)
        train.expert_linear_backward_input(d_logits, W["router"], dx_router, status=st)
        return dx + dx_router, d_w, d_logits, grads

    def check(self):
        for status in (self.moe.get_error(), int(self.status)):
            if status != moe.MOE_OK:
                raise moe.MoEError(status, "expert layer")


def run(tokens, hidden, inter, shared, experts, top_k, seed=0):
    """One step on random tokens: (the layer, its input, the gradient of its output, its output, gradients)."""
    layer = ExpertLayer(tokens, hidden, inter, shared, experts, top_k, seed)
    g = torch.Generator(device="cuda").manual_seed(seed + 1)
    x, d_out = (torch.randn(tokens, hidden, generator=g, **BF16) for _ in range(2))
    out = layer.forward(x)
    grads = layer.backward(d_out)
    layer.check()
    return layer, x, d_out, out, grads


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--tokens", type=int, default=4096)
    ap.add_argument("--hidden", type=int, default=4096)
    ap.add_argument("--inter", type=int, default=2048)
    ap.add_argument("--shared", type=int, default=2048)
    ap.add_argument("--experts", type=int, default=32)
    ap.add_argument("--top-k", type=int, default=4)
    a = ap.parse_args()
    layer, x, d_out, _, _ = run(a.tokens, a.hidden, a.inter, a.shared, a.experts, a.top_k)
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    start.record()
    for _ in range(5):
        layer.forward(x)
        layer.backward(d_out)
    end.record()
    end.synchronize()
    flops = 18 * a.tokens * a.hidden * (a.top_k * a.inter + a.shared)
    ms = start.elapsed_time(end) / 5
    print(f"{a.tokens} tokens through {a.top_k} of {a.experts} experts and a shared one: {ms:.2f} ms a step, "
          f"{flops / ms / 1e9:.0f} TFLOP/s")


if __name__ == "__main__":
    main()
