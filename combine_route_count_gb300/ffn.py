"""The feed-forward operators of include/moe_ffn.h on torch tensors.

Each function checks its tensors (type, shape, contiguity, device), then makes
one call into libmoe.so on the given stream (torch's current stream if None).
Outputs are the caller's tensors, as everywhere in this package; nothing is
allocated and nothing waits for the GPU.  E4M3 codes may be given as
``torch.float8_e4m3fn`` or as their ``torch.uint8`` bytes.  A wrong argument
raises ``moe.MoEError`` with ``MOE_EINVAL`` before anything is enqueued.
"""
from __future__ import annotations

from typing import Any, Optional

import torch

from . import moe

BLOCK = moe.MOE_FP8_BLOCK

_FP8 = (torch.float8_e4m3fn, torch.uint8)
_BF16 = (torch.bfloat16, torch.int16)  # int16: the bits, as the dispatch and combine calls take them
_F32 = (torch.float32,)
_FLOAT = (torch.bfloat16, torch.float32)


def _wrong(what: str) -> "moe.MoEError":
    return moe.MoEError(moe.MOE_EINVAL, what)


def _arg(name: str, t: Any, dtypes: tuple, shape: tuple, device: Any) -> int:
    """The tensor's address; raises unless it is what the call takes."""
    if not isinstance(t, torch.Tensor):
        raise _wrong(f"{name} must be a tensor")
    if t.dtype not in dtypes:
        raise _wrong(f"{name} has type {t.dtype}, must be {' or '.join(map(str, dtypes))}")
    if t.shape != shape:
        raise _wrong(f"{name} has shape {tuple(t.shape)}, must be {tuple(shape)}")
    if not t.is_contiguous():
        raise _wrong(f"{name} must be contiguous")
    if t.device != device:
        raise _wrong(f"{name} is on {t.device}, must be on {device}")
    return t.data_ptr()


def _device(name: str, t: Any, ndim: int) -> Any:
    """The device the call runs on: the first tensor's, which must be current."""
    if not isinstance(t, torch.Tensor) or t.dim() != ndim:
        raise _wrong(f"{name} must be a tensor of {ndim} dimensions")
    if not t.is_cuda or t.get_device() != torch.cuda.current_device():
        raise _wrong(f"{name} must be on the current CUDA device")
    return t.device


def add_rms_norm_fp8(x: torch.Tensor, weight: torch.Tensor, xq: torch.Tensor, x_scales: torch.Tensor, *,
                     eps: float = 1e-6, residual: Optional[torch.Tensor] = None,
                     residual_out: Optional[torch.Tensor] = None, y: Optional[torch.Tensor] = None,
                     stream: Any = None) -> None:
    """Residual addition, RMS norm and quantisation of token rows.

    x bf16 [T, H] (H a multiple of 128), weight bf16 or float32 [H]; writes
    xq E4M3 [T, H] and x_scales float32 [T, H/128], the payload that
    ``MoELayer.dispatch_send_quantized`` and ``DecodeLayer`` take.  residual
    bf16 [T, H] is added first, the sum goes to residual_out (may be x or
    residual); y bf16 [T, H], if given, receives the normalised rows."""
    dev = _device("x", x, 2)
    T, H = x.shape
    px = _arg("x", x, _BF16, (T, H), dev)
    pw = _arg("weight", weight, _FLOAT, (H,), dev)
    pq = _arg("xq", xq, _FP8, (T, H), dev)
    ps = _arg("x_scales", x_scales, _F32, (T, H // BLOCK), dev)
    if (residual is None) != (residual_out is None):
        raise _wrong("residual and residual_out go together")
    pr = po = py = None
    if residual is not None:
        pr = _arg("residual", residual, _BF16, (T, H), dev)
        po = _arg("residual_out", residual_out, _BF16, (T, H), dev)
    if y is not None:
        py = _arg("y", y, _BF16, (T, H), dev)
    moe.moe_add_rms_norm_fp8(px, pr, pw, moe.MOE_TYPE_F32 if weight.dtype == torch.float32 else moe.MOE_TYPE_BF16,
                             T, H, eps, po, py, pq, ps, stream)
