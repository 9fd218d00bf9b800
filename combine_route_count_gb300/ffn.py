"""The feed-forward operators of include/moe_ffn.h on torch tensors.

Each function checks its tensors (type, shape, contiguity, device), then makes
one call into libmoe.so on the given stream (torch's current stream if None).
Outputs are the caller's tensors, as everywhere in this package; the functions
allocate nothing and nothing waits for the GPU.  E4M3 codes may be given as
``torch.float8_e4m3fn`` or as their ``torch.uint8`` bytes, bf16 rows also as
``torch.int16`` bits.  A wrong argument raises ``moe.MoEError`` with
``MOE_EINVAL`` before anything is enqueued.

``DecodeLayer`` keeps one layer's weights and the workspace of its calls.

The checks run in the CPython module ``_ffn`` (csrc/ffn_py.cc), built next to
libmoe.so; there is no fallback: if it is missing, every call raises.
"""
from __future__ import annotations

import importlib
import os
import struct
import threading
from typing import Any, Optional

import torch

from . import moe

BLOCK = moe.MOE_FP8_BLOCK

_module: Any = None
# The current stream's handle without a stream object.
_raw_stream = torch._C._cuda_getCurrentRawStream


def _native() -> Any:
    global _module
    if _module is None:
        path = os.path.join(moe.PKG, "_ffn.so")
        if not os.path.exists(path):
            raise RuntimeError(f"_ffn.so is not built ({path}); run __graft_entry__.build() "
                               "or python combine_route_count_gb300/build.py")
        moe.load_library()
        module = importlib.import_module("._ffn", __package__)
        module.init(moe.MoEError)
        _module = module
    return _module


def _stream(stream: Any, t: Any) -> int:
    if stream is None:
        # The call checks that the tensor is on the current device.
        return _raw_stream(t.get_device()) if isinstance(t, torch.Tensor) and t.is_cuda else 0
    return moe._stream(stream) or 0


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
    (_module or _native()).add_rms_norm_fp8(x, weight, xq, x_scales, eps, residual, residual_out, y,
                                            _stream(stream, x))


def expert_gemm_fp8(a: torch.Tensor, a_scales: torch.Tensor, w: torch.Tensor, w_scales: torch.Tensor,
                    out: torch.Tensor, *, expert_offsets: Optional[torch.Tensor] = None,
                    status: Optional[torch.Tensor] = None, stream: Any = None) -> None:
    """out[i] = a[i] . w[e]^T for the rows i that expert_offsets gives expert e.

    a E4M3 [rows, K] with a_scales float32 [rows, ceil(K/128)]; w E4M3
    [E, N, K] with w_scales float32 [E, ceil(N/128), ceil(K/128)] (or both
    without the first dimension for one expert); out bf16 or float32 [rows, N].
    expert_offsets int32 [E+1], e.g. ``dispatch_recv()["expert_offsets"]``;
    None for one expert with all rows.  K % 16 == 0, N % 8 == 0.  status int32
    [1], which the caller sets to MOE_OK, becomes MOE_ETIMEDOUT if a wait inside
    the kernel gives up; without one, incomplete rows are not reported."""
    (_module or _native()).expert_product(False, a, a_scales, w, w_scales, out, None, expert_offsets, status,
                                          _stream(stream, a))


def expert_glu_fp8(a: torch.Tensor, a_scales: torch.Tensor, w13: torch.Tensor, w13_scales: torch.Tensor,
                   hq: torch.Tensor, h_scales: torch.Tensor, *, expert_offsets: Optional[torch.Tensor] = None,
                   status: Optional[torch.Tensor] = None, stream: Any = None) -> None:
    """h = SiLU(a . gate^T) * (a . up^T), quantised: the rows of the second product.

    As expert_gemm_fp8 (status too), with w13 [E, 2*I, H] (gate rows, then up rows; I a
    multiple of 128); hq E4M3 [rows, I], h_scales float32 [rows, I/128]."""
    (_module or _native()).expert_product(True, a, a_scales, w13, w13_scales, hq, h_scales, expert_offsets, status,
                                          _stream(stream, a))


class DecodeLayer:
    """A whole expert layer for a few tokens, for one layer's weights.

    Keeps references to the weights (w13 E4M3 [E, 2*I, H], gate rows then up
    rows; w2 E4M3 [E, H, I]; their scales float32 [E, 2*I/128, H/128] and
    [E, H/128, I/128]) and owns the workspace for up to max_tokens tokens of
    top_k experts.  Every call reads the weights where the tensors then have
    them: they may be overwritten, or given other storage of the same shape,
    between calls.  Calls may be on any stream, also on another than the one
    the layer was built on, but only one may be in flight at a time: calls that
    may overlap need a layer object each (calls of several threads on one stream
    do not overlap).  Building a layer waits for the
    current stream.  A layer may be dropped while a call is in flight; one that
    is part of a CUDA graph has to live as long as the graph."""

    def __init__(self, max_tokens: int, top_k: int, w13: torch.Tensor, w13_scales: torch.Tensor, w2: torch.Tensor,
                 w2_scales: torch.Tensor):
        wrong = lambda what: moe.MoEError(moe.MOE_EINVAL, what)  # noqa: E731
        for name, t in (("w13", w13), ("w2", w2)):
            if not isinstance(t, torch.Tensor) or t.dim() != 3:
                raise wrong(f"{name} must be a tensor of 3 dimensions")
        if not w13.is_cuda or w13.get_device() != torch.cuda.current_device():
            raise wrong("w13 must be on the current CUDA device")
        self.E, self.H, self.I = w2.shape
        self.max_tokens, self.K, self.device = max_tokens, top_k, w13.device
        E, H, I, dev = self.E, self.H, self.I, self.device.index
        self._weights = (w13, w13_scales, w2, w2_scales)
        _native().check_weights(self._weights, E, H, I, dev)
        nbytes = moe.moe_decode_workspace_bytes(moe.make_config(max_tokens, H, top_k, E, 1), I)
        self.workspace = torch.empty(max(nbytes, 256), dtype=torch.uint8, device=self.device)
        self.status = torch.zeros(1, dtype=torch.int32, device=self.device)
        self._streams = {_raw_stream(dev)}
        self._lock = threading.Lock()  # a call is two launches, made without the interpreter lock
        if not torch.cuda.is_current_stream_capturing():
            # What this stream still does with the new blocks (the zero; their
            # users before) is over before a call on another stream writes them.
            torch.cuda.current_stream().synchronize()
        self._plan = struct.pack("6i3Q", max_tokens, H, top_k, E, I, dev, self.status.data_ptr(),
                                 self.workspace.data_ptr(), self.workspace.numel())

    def forward(self, xq: torch.Tensor, x_scales: torch.Tensor, topk_idx: torch.Tensor, topk_w: torch.Tensor,
                out: torch.Tensor, stream: Any = None) -> None:
        """out[t] = sum_k topk_w[t,k] * expert(topk_idx[t,k])(x[t]); out bf16 [T, H], T <= max_tokens."""
        handle = _stream(stream, xq)
        with self._lock:
            if handle not in self._streams:
                self._use_on(handle)
            _module.decode_layer_fp8(self._plan, self._weights, xq, x_scales, topk_idx, topk_w, out, handle)

    def _use_on(self, handle: int) -> None:
        """Memory that is freed with the layer is not given to others before this stream is done with it."""
        stream = torch.cuda.ExternalStream(handle, device=self.device)
        for t in (self.workspace, self.status, *self._weights):
            t.record_stream(stream)
        self._streams.add(handle)

    def get_error(self, stream: Any = None) -> int:
        """Waits for the stream (given as to forward); the device status of the last call that had tokens.

        MOE_OK, MOE_EROUTE or MOE_ETIMEDOUT; MOE_OK before the first such call."""
        torch.cuda.ExternalStream(_stream(stream, self.status), device=self.device).synchronize()
        return int(self.status.item())
