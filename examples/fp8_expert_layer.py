"""One fp8 expert layer end to end on one GPU, by both of its ways.

Many tokens: residual + RMS norm + quantisation, dispatch of the quantised rows,
the experts' gate/up product with SiLU and requantisation, their second
product, and the weighted combine.  A few tokens: the same norm, then the whole
layer in two kernels.  Weights and tokens are random; the two ways are compared
on the first tokens.

    python examples/fp8_expert_layer.py [--tokens 4096] [--few 16]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from combine_route_count_gb300 import ffn, moe  # noqa: E402

FP8 = torch.float8_e4m3fn


class ExpertLayer:
    """Weights of one layer and the buffers of its two ways."""

    def __init__(self, tokens, few, hidden, inter, experts, top_k, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.H, self.I, self.E, self.K = hidden, inter, experts, top_k

        def weights(n, k):
            w = (torch.randn(experts, n, k, generator=g, device="cuda", dtype=torch.bfloat16) * 107).clamp_(-448, 448)
            s = (0.5 + torch.rand(experts, n // 128, k // 128, generator=g, device="cuda")) / (107.0 * k ** 0.5)
            return w.to(FP8), s

        self.w13, self.s13 = weights(2 * inter, hidden)
        self.w2, self.s2 = weights(hidden, inter)
        self.norm = torch.ones(hidden, dtype=torch.bfloat16, device="cuda")
        self.router = torch.randn(experts, hidden, generator=g, device="cuda", dtype=torch.bfloat16)
        self.moe = moe.MoELayer(tokens, hidden, top_k, experts, 1)
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")  # of the products
        self.decode = ffn.DecodeLayer(few, top_k, self.w13, self.s13, self.w2, self.s2)

    def normalise(self, x, residual):
        """The layer's input: rows for the router, codes for the experts; residual is updated in place."""
        T, H = x.shape
        y, q = torch.empty_like(x), torch.empty(T, H, dtype=FP8, device=x.device)
        scales = torch.empty(T, H // 128, device=x.device)
        ffn.add_rms_norm_fp8(x, self.norm, q, scales, residual=residual, residual_out=residual, y=y)
        return y, q, scales

    def route(self, y):
        weight, idx = torch.topk(torch.softmax((y @ self.router.t()).float(), 1), self.K, 1)
        return idx.to(torch.int32), weight / weight.sum(1, keepdim=True)

    def forward_many(self, q, scales, idx, weight):
        T = q.shape[0]
        rows, dev = T * self.K, q.device
        ex, es = torch.empty(rows, self.H, dtype=FP8, device=dev), torch.empty(rows, self.H // 128, device=dev)
        self.moe.dispatch_send_quantized(q, scales, idx, ex, es)
        offsets = self.moe.dispatch_recv()["expert_offsets"]
        hq, hs = torch.empty(rows, self.I, dtype=FP8, device=dev), torch.empty(rows, self.I // 128, device=dev)
        ffn.expert_glu_fp8(ex, es, self.w13, self.s13, hq, hs, expert_offsets=offsets, status=self.status)
        y = torch.empty(rows, self.H, dtype=torch.bfloat16, device=dev)
        ffn.expert_gemm_fp8(hq, hs, self.w2, self.s2, y, expert_offsets=offsets, status=self.status)
        out = torch.empty(T, self.H, dtype=torch.bfloat16, device=dev)
        self.moe.combine_send(y)
        self.moe.combine_recv(weight, out)
        return out

    def forward_few(self, q, scales, idx, weight):
        out = torch.empty(q.shape[0], self.H, dtype=torch.bfloat16, device=q.device)
        self.decode.forward(q, scales, idx, weight, out)
        return out


def run(tokens, few, hidden, inter, experts, top_k, seed=0):
    """Runs both ways on the same tokens; returns (out of many, out of the first few)."""
    layer = ExpertLayer(tokens, few, hidden, inter, experts, top_k, seed)
    g = torch.Generator(device="cuda").manual_seed(seed + 1)
    x = torch.randn(tokens, hidden, generator=g, device="cuda", dtype=torch.bfloat16)
    residual = torch.randn(tokens, hidden, generator=g, device="cuda", dtype=torch.bfloat16)
    y, q, scales = layer.normalise(x, residual)
    idx, weight = layer.route(y)
    many = layer.forward_many(q, scales, idx, weight)
    part = layer.forward_few(q[:few], scales[:few], idx[:few], weight[:few])
    for status in (layer.moe.get_error(), int(layer.status), layer.decode.get_error()):
        if status != moe.MOE_OK:
            raise moe.MoEError(status, "expert layer")
    return many, part


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--tokens", type=int, default=4096)
    ap.add_argument("--few", type=int, default=16)
    ap.add_argument("--hidden", type=int, default=7168)
    ap.add_argument("--inter", type=int, default=2048)
    ap.add_argument("--experts", type=int, default=64)
    ap.add_argument("--top-k", type=int, default=8)
    a = ap.parse_args()
    many, part = run(a.tokens, a.few, a.hidden, a.inter, a.experts, a.top_k)
    far = (many[: a.few].float() - part.float()).norm() / part.float().norm()
    print(f"{a.tokens} tokens through {a.experts} experts; the first {a.few} both ways: relative difference {far:.4f}")


if __name__ == "__main__":
    main()
