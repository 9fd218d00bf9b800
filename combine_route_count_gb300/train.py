"""The training operators of include/moe_train.h on torch tensors.

The router, the bf16 expert products and the gradients of dispatch, products and
combine.  As in ``ffn``: each function checks its tensors (type, shape,
contiguity, device), then makes one call into libmoe.so on the given stream
(torch's current stream if None).  Outputs are the caller's tensors, the
functions allocate nothing and nothing waits for the GPU.  bf16 rows may be given
as ``torch.int16`` bits too.  A wrong argument raises ``moe.MoEError`` with
``MOE_EINVAL`` before anything is enqueued.

A training step of one layer, with ``lay = layer.dispatch_recv()``:

    router_topk(logits, idx, w);  layer.dispatch_send(x, idx, expert_x)
    expert_linear(expert_x, w13, h, activation="swiglu", pre=pre, expert_offsets=lay["expert_offsets"])
    expert_linear(h, w2, expert_y, expert_offsets=lay["expert_offsets"])
    layer.combine_send(expert_y);  layer.combine_recv(w, out)

    combine_backward(d_out, lay["slot_row"], w, d_y, expert_y=expert_y, d_topk_w=d_w)
    expert_linear_backward_weight(d_y, h, d_w2, expert_offsets=lay["expert_offsets"])
    expert_linear_backward_input(d_y, w2, d_pre, activation="swiglu", pre=pre, expert_offsets=lay["expert_offsets"])
    expert_linear_backward_weight(d_pre, expert_x, d_w13, expert_offsets=lay["expert_offsets"])
    expert_linear_backward_input(d_pre, w13, d_expert_x, expert_offsets=lay["expert_offsets"])
    dispatch_backward(d_expert_x, lay["slot_row"], d_x);  router_topk_backward(logits, idx, d_w, d_logits)

The layout's arrays live in the layer's workspace until its next dispatch_send.

The checks run in the CPython module ``_train`` (csrc/train_py.cc), built next to
libmoe.so; there is no fallback: if it is missing, every call raises.
"""
from __future__ import annotations

import importlib
import os
from typing import Any, Optional

import torch

from . import ffn, moe

SCORES = {"softmax": moe.MOE_SCORE_SOFTMAX, "sigmoid": moe.MOE_SCORE_SIGMOID}
ACTIVATIONS = {"none": moe.MOE_ACT_NONE, "relu": moe.MOE_ACT_RELU, "gelu": moe.MOE_ACT_GELU,
               "silu": moe.MOE_ACT_SILU, "swiglu": moe.MOE_ACT_SWIGLU}


_module: Any = None


def _native() -> Any:
    global _module
    if _module is None:
        path = os.path.join(moe.PKG, "_train.so")
        if not os.path.exists(path):
            raise RuntimeError(f"_train.so is not built ({path}); run __graft_entry__.build() "
                               "or python combine_route_count_gb300/build.py")
        moe.load_library()
        module = importlib.import_module("._train", __package__)
        module.init(moe.MoEError)
        _module = module
    return _module


def _named(what: str, names: dict, name: str) -> int:
    try:
        return names[name]
    except (KeyError, TypeError):
        raise moe.MoEError(moe.MOE_EINVAL, f"{what} must be one of {', '.join(names)}") from None


def router_topk(logits: torch.Tensor, topk_idx: torch.Tensor, topk_w: torch.Tensor, *, score: str = "softmax",
                bias: Optional[torch.Tensor] = None, normalize: bool = True, scale: float = 1.0,
                stream: Any = None) -> None:
    """Chooses each token's experts and their weights.

    logits bf16 or float32 [T, E]; writes topk_idx int32 [T, K], the experts
    with the largest score (plus bias float32 [E], which only "sigmoid" takes),
    the lower index first among equals, and topk_w float32 [T, K] = scale *
    score, with normalize divided by the sum over the token's choices."""
    (_module or _native()).router_topk(logits, topk_idx, topk_w, bias, _named("score", SCORES, score),
                                               normalize, scale, ffn._stream(stream, logits))


def router_topk_backward(logits: torch.Tensor, topk_idx: torch.Tensor, d_topk_w: torch.Tensor,
                         d_logits: torch.Tensor, *, score: str = "softmax", normalize: bool = True,
                         scale: float = 1.0, stream: Any = None) -> None:
    """Gradient of router_topk's weights by the logits, the choice held fixed.

    d_topk_w float32 [T, K]; writes d_logits [T, E] of the logits' type, all of it."""
    (_module or _native()).router_topk_backward(logits, topk_idx, d_topk_w, d_logits,
                                                        _named("score", SCORES, score), normalize, scale,
                                                        ffn._stream(stream, logits))


def combine_backward(d_out: torch.Tensor, slot_row: torch.Tensor, topk_w: torch.Tensor, d_expert_y: torch.Tensor, *,
                     expert_y: Optional[torch.Tensor] = None, d_topk_w: Optional[torch.Tensor] = None,
                     stream: Any = None) -> None:
    """Gradient of ``MoELayer.combine_recv``.

    d_out bf16 [T, H], slot_row int32 [T, K] of the dispatch's layout, topk_w
    float32 [T, K]; writes the rows of d_expert_y bf16 [rows, H] that slot_row
    names (may be expert_y itself) and, from expert_y bf16 [rows, H], d_topk_w
    float32 [T, K] (both or neither)."""
    (_module or _native()).combine_backward(d_out, slot_row, topk_w, d_expert_y, expert_y, d_topk_w,
                                                    ffn._stream(stream, d_out))


def dispatch_backward(d_expert_x: torch.Tensor, slot_row: torch.Tensor, d_x: torch.Tensor, *,
                      add: Optional[torch.Tensor] = None, stream: Any = None) -> None:
    """Gradient of ``MoELayer.dispatch_send``: d_x[t] = sum_k d_expert_x[slot_row[t, k]] (+ add[t]).

    d_expert_x bf16 [rows, H], d_x and add bf16 [T, H] (add may be d_x)."""
    (_module or _native()).dispatch_backward(d_expert_x, slot_row, d_x, add, ffn._stream(stream, d_expert_x))


def expert_linear(a: torch.Tensor, w: torch.Tensor, out: torch.Tensor, *, bias: Optional[torch.Tensor] = None,
                  activation: str = "none", residual: Optional[torch.Tensor] = None,
                  pre: Optional[torch.Tensor] = None, expert_offsets: Optional[torch.Tensor] = None,
                  status: Optional[torch.Tensor] = None, stream: Any = None) -> None:
    """out[i] = act(a[i] . w[e]^T + bias[e]) + residual[i] for the rows i that expert_offsets gives expert e.

    a bf16 [rows, K], w bf16 [E, N, K] (or [N, K] for one expert), bias bf16 or
    float32 [E, N], activation "none", "relu", "gelu", "silu" or "swiglu" (w's
    first N/2 rows are the gate's), residual bf16 and out bf16 or float32
    [rows, N] (swiglu: [rows, N/2]), pre bf16 [rows, N]: what the activation was
    taken of.  expert_offsets int32 [E+1], None for one expert with all rows.
    K % 8 == 0, N % 8 == 0.  status as for ``ffn.expert_gemm_fp8``."""
    (_module or _native()).expert_linear(a, w, out, bias, _named("activation", ACTIVATIONS, activation),
                                                 residual, pre, expert_offsets, status, ffn._stream(stream, a))


def expert_linear_backward_input(dy: torch.Tensor, w: torch.Tensor, dx: torch.Tensor, *, activation: str = "none",
                                 pre: Optional[torch.Tensor] = None, expert_offsets: Optional[torch.Tensor] = None,
                                 status: Optional[torch.Tensor] = None, stream: Any = None) -> None:
    """dx[i] = (dy[i] . w[e]) * act'(pre[i]), the gradient by a product's rows, on through the activation they came from.

    dy bf16 [rows, N], w bf16 [E, N, K], dx and pre bf16 [rows, K] ("swiglu":
    [rows, 2K], gate and up); dx may be pre.  "none" (without pre): dx = dy . w."""
    (_module or _native()).expert_linear_backward_input(
        dy, w, dx, _named("activation", ACTIVATIONS, activation), pre, expert_offsets, status, ffn._stream(stream, dy))


def expert_linear_backward_weight(dy: torch.Tensor, a: torch.Tensor, dw: torch.Tensor, *,
                                  db: Optional[torch.Tensor] = None, accumulate: bool = False,
                                  expert_offsets: Optional[torch.Tensor] = None,
                                  status: Optional[torch.Tensor] = None, stream: Any = None) -> None:
    """dw[e] = dy_e^T . a_e and db[e] = the sum of dy_e over expert e's rows; added to them with accumulate.

    dy bf16 [rows, N], a bf16 [rows, K], dw bf16 or float32 [E, N, K], db float32 [E, N]."""
    (_module or _native()).expert_linear_backward_weight(dy, a, dw, db, accumulate, expert_offsets, status,
                                                                 ffn._stream(stream, dy))
