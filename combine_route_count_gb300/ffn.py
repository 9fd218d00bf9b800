"""The feed-forward operators of include/moe_ffn.h on torch tensors.

Each function checks its tensors (type, shape, contiguity, device), then makes
one call into libmoe.so on the given stream (torch's current stream if None).
Outputs are the caller's tensors, as everywhere in this package; the functions
allocate nothing and nothing waits for the GPU.  E4M3 codes may be given as
``torch.float8_e4m3fn`` or as their ``torch.uint8`` bytes.  A wrong argument
raises ``moe.MoEError`` with ``MOE_EINVAL`` before anything is enqueued.

``DecodeLayer`` keeps one layer's weights and the workspace of its calls.
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


# The calls are often launch-bound, so their checks are kept to a few attribute
# reads per tensor: the raw stream and device queries below are what
# torch.cuda.current_stream() and current_device() return, without the objects.
_raw_stream = torch._C._cuda_getCurrentRawStream
_current_device = torch._C._cuda_getDevice


def _wrong(what: str) -> "moe.MoEError":
    return moe.MoEError(moe.MOE_EINVAL, what)


def _arg(name: str, t: torch.Tensor, dtypes: tuple, shape: tuple, device: int) -> int:
    """The tensor's address; raises unless it is what the call takes."""
    try:
        if t.dtype in dtypes and t.shape == shape and t.is_contiguous() and t.get_device() == device:
            return t.data_ptr()
    except (AttributeError, TypeError):
        raise _wrong(f"{name} must be a tensor") from None
    if t.dtype not in dtypes:
        raise _wrong(f"{name} has type {t.dtype}, must be {' or '.join(map(str, dtypes))}")
    if t.shape != shape:
        raise _wrong(f"{name} has shape {tuple(t.shape)}, must be {tuple(shape)}")
    if not t.is_contiguous():
        raise _wrong(f"{name} must be contiguous")
    raise _wrong(f"{name} is on {t.device}, must be on cuda:{device}")


def _device(name: str, t: Any, ndim: int) -> int:
    """The device the call runs on: the first tensor's, which must be current."""
    if not isinstance(t, torch.Tensor) or t.dim() != ndim:
        raise _wrong(f"{name} must be a tensor of {ndim} dimensions")
    if not t.is_cuda or t.get_device() != _current_device():
        raise _wrong(f"{name} must be on the current CUDA device")
    return t.get_device()


def _stream(stream: Any, device: int) -> int:
    return _raw_stream(device) if stream is None else moe._stream(stream)


def _lib() -> Any:
    return moe._lib or moe.load_library()


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
    rc = _lib().moe_add_rms_norm_fp8(px, pr, pw, weight.dtype == torch.float32, T, H, eps, po, py, pq, ps,
                                     _stream(stream, dev))
    if rc:
        raise moe.MoEError(rc, "moe_add_rms_norm_fp8")


def _blocks(n: int) -> int:
    return (n + BLOCK - 1) // BLOCK


def _product_args(a, a_scales, w, w_scales, expert_offsets, status):
    """The checks that the two products share; w may be [N, K] for one expert."""
    dev = _device("a", a, 2)
    rows, K = a.shape
    if not isinstance(w, torch.Tensor) or w.dim() not in (2, 3):
        raise _wrong("w must be a tensor of 3 dimensions, or 2 for one expert")
    experts = () if w.dim() == 2 else (w.shape[0],)
    E, N = (1, w.shape[0]) if w.dim() == 2 else w.shape[:2]
    pa = _arg("a", a, _FP8, (rows, K), dev)
    ps = _arg("a_scales", a_scales, _F32, (rows, _blocks(K)), dev)
    pw = _arg("w", w, _FP8, (*experts, N, K), dev)
    pv = _arg("w_scales", w_scales, _F32, (*experts, _blocks(N), _blocks(K)), dev)
    po = None if expert_offsets is None else _arg("expert_offsets", expert_offsets, (torch.int32,), (E + 1,), dev)
    pt = None if status is None else _arg("status", status, (torch.int32,), (1,), dev)
    return dev, rows, K, N, E, pa, ps, pw, pv, po, pt


def expert_gemm_fp8(a: torch.Tensor, a_scales: torch.Tensor, w: torch.Tensor, w_scales: torch.Tensor,
                    out: torch.Tensor, *, expert_offsets: Optional[torch.Tensor] = None,
                    status: Optional[torch.Tensor] = None, stream: Any = None) -> None:
    """out[i] = a[i] . w[e]^T for the rows i that expert_offsets gives expert e.

    a E4M3 [rows, K] with a_scales float32 [rows, ceil(K/128)]; w E4M3
    [E, N, K] with w_scales float32 [E, ceil(N/128), ceil(K/128)]; out bf16 or
    float32 [rows, N].  expert_offsets int32 [E+1], e.g.
    ``dispatch_recv()["expert_offsets"]``; None for one expert with all rows.
    K % 16 == 0, N % 8 == 0."""
    dev, rows, K, N, E, pa, ps, pw, pv, po, pt = _product_args(a, a_scales, w, w_scales, expert_offsets, status)
    pout = _arg("out", out, _FLOAT, (rows, N), dev)
    rc = _lib().moe_expert_gemm_fp8(pa, ps, rows, K, pw, pv, N, E, po, pout, out.dtype == torch.float32, pt,
                                    _stream(stream, dev))
    if rc:
        raise moe.MoEError(rc, "moe_expert_gemm_fp8")


def expert_glu_fp8(a: torch.Tensor, a_scales: torch.Tensor, w13: torch.Tensor, w13_scales: torch.Tensor,
                   hq: torch.Tensor, h_scales: torch.Tensor, *, expert_offsets: Optional[torch.Tensor] = None,
                   status: Optional[torch.Tensor] = None, stream: Any = None) -> None:
    """h = SiLU(a . gate^T) * (a . up^T), quantised: the rows of the second product.

    As expert_gemm_fp8, with w13 [E, 2*I, H] (gate rows, then up rows; I a
    multiple of 128); hq E4M3 [rows, I], h_scales float32 [rows, I/128]."""
    dev, rows, H, N, E, pa, ps, pw, pv, po, pt = _product_args(a, a_scales, w13, w13_scales, expert_offsets, status)
    if N % (2 * BLOCK):
        raise _wrong(f"w13 has {N} rows, must be twice a multiple of {BLOCK}")
    I = N // 2
    ph = _arg("hq", hq, _FP8, (rows, I), dev)
    pg = _arg("h_scales", h_scales, _F32, (rows, I // BLOCK), dev)
    rc = _lib().moe_expert_glu_fp8(pa, ps, rows, H, pw, pv, I, E, po, ph, pg, pt, _stream(stream, dev))
    if rc:
        raise moe.MoEError(rc, "moe_expert_glu_fp8")


class DecodeLayer:
    """A whole expert layer for a few tokens, for one layer's weights.

    Keeps references to the weights (w13 E4M3 [E, 2*I, H], gate rows then up
    rows; w2 E4M3 [E, H, I]; their scales float32 [E, 2*I/128, H/128] and
    [E, H/128, I/128]) and owns the workspace for up to max_tokens tokens of
    top_k experts.  One call may be in flight at a time: calls on several
    streams need a layer object each."""

    def __init__(self, max_tokens: int, top_k: int, w13: torch.Tensor, w13_scales: torch.Tensor, w2: torch.Tensor,
                 w2_scales: torch.Tensor):
        dev = _device("w13", w13, 3)
        self.device = w13.device
        if not isinstance(w2, torch.Tensor) or w2.dim() != 3:
            raise _wrong("w2 must be a tensor of 3 dimensions")
        self.E, self.H, self.I = w2.shape
        self.max_tokens, self.K = max_tokens, top_k
        self._weights = (w13, w13_scales, w2, w2_scales)  # kept alive; their addresses are passed on
        sizes = ("w13", w13, _FP8, (self.E, 2 * self.I, self.H)), \
                ("w13_scales", w13_scales, _F32, (self.E, _blocks(2 * self.I), _blocks(self.H))), \
                ("w2", w2, _FP8, (self.E, self.H, self.I)), \
                ("w2_scales", w2_scales, _F32, (self.E, _blocks(self.H), _blocks(self.I)))
        self._pointers = tuple(_arg(*s, dev) for s in sizes)
        self._config = moe.make_config(max_tokens, self.H, top_k, self.E, 1)
        nbytes = moe.moe_decode_workspace_bytes(self._config, self.I)
        self.workspace = torch.empty(max(nbytes, 256), dtype=torch.uint8, device=self.device)
        self.status = torch.zeros(1, dtype=torch.int32, device=self.device)
        self._own = (self.status.data_ptr(), self.workspace.data_ptr(), self.workspace.numel())

    def forward(self, xq: torch.Tensor, x_scales: torch.Tensor, topk_idx: torch.Tensor, topk_w: torch.Tensor,
                out: torch.Tensor, stream: Any = None) -> None:
        """out[t] = sum_k topk_w[t,k] * expert(topk_idx[t,k])(x[t]); out bf16 [T, H], T <= max_tokens."""
        dev = _device("xq", xq, 2)
        T, H, K = xq.shape[0], self.H, self.K
        if T > self.max_tokens or dev != self.device.index:
            raise _wrong(f"xq has {T} tokens on cuda:{dev}, must have at most {self.max_tokens} on {self.device}")
        px = _arg("xq", xq, _FP8, (T, H), dev)
        ps = _arg("x_scales", x_scales, _F32, (T, H // BLOCK), dev)
        pi = _arg("topk_idx", topk_idx, (torch.int32,), (T, K), dev)
        pw = _arg("topk_w", topk_w, _F32, (T, K), dev)
        po = _arg("out", out, _BF16, (T, H), dev)
        self._config.num_tokens = T
        rc = _lib().moe_decode_layer_fp8(self._config, self.I, px, ps, pi, pw, *self._pointers, po, *self._own,
                                         _stream(stream, dev))
        if rc:
            raise moe.MoEError(rc, "moe_decode_layer_fp8")

    def get_error(self, stream: Any = None) -> int:
        """Waits for the stream; the device status of the last call (MOE_OK or MOE_EROUTE)."""
        s = torch.cuda.current_stream() if stream is None else stream
        s.synchronize()
        return int(self.status.item())
