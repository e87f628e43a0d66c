"""The dense operators around the routed experts, on torch tensors.

``rms_norm`` adds the residual, normalises and quantises in one pass,
``quantize_fp8`` makes the same 8-bit form of given rows, ``linear`` is a
matrix product with bias, activation (plain or gated) and residual in its
epilogue, on bf16, fp16 or 8-bit operands.  A dense feed-forward beside the
experts, in 8 bits end to end:

    n = rms_norm(x, weight, residual=h, scales="mx")       # n.y: the experts' bf16 input
    logits = linear(n.y, w_router, out_dtype=torch.float32)
    a = linear(n.fp8, w_gate_up, act="gelu_tanh", gated=True, out_dtype="mx")
    out = linear(a, w_down, residual=n.total)

All functions raise ValueError for tensors of the wrong dtype, shape, layout
or device, queue their work on `stream` (torch's current stream of the
tensors' device when None; an integer is a raw HIP stream handle) and return
without waiting.  They allocate through torch, so they can be captured into a
graph.  Forward only: no gradients are recorded.
"""
from __future__ import annotations

import ctypes
import operator
from typing import NamedTuple, Optional, Union

import torch

from . import _lib

_TYPES = {torch.bfloat16: _lib.TYPE_BF16, torch.float16: _lib.TYPE_FP16,
          torch.float32: _lib.TYPE_FP32}
_FP8 = {"row": _lib.TYPE_FP8_ROW, "mx": _lib.TYPE_FP8_MX}
_ACTS = {None: _lib.ACT_NONE, "none": _lib.ACT_NONE, "silu": _lib.ACT_SILU,
         "gelu": _lib.ACT_GELU, "gelu_tanh": _lib.ACT_GELU_TANH, "relu": _lib.ACT_RELU}


class FP8Rows(NamedTuple):
    """Rows held in 8 bits: E4M3 codes uint8 [rows, K] and their scales, fp32
    [rows] ("row") or UE8M0 uint8 [rows, K/32] ("mx").  Where an FP8Rows is
    taken, any (codes, scales) pair is."""
    codes: torch.Tensor
    scales: torch.Tensor

    def dequantize(self) -> torch.Tensor:
        """The values, in fp32 (with torch operations)."""
        v = self.codes.view(torch.float8_e4m3fn).float()
        if self.scales.dtype == torch.float32:
            return v * self.scales[:, None]
        s = self.scales.view(torch.float8_e8m0fnu).float()
        return (v.view(v.shape[0], -1, 32) * s[..., None]).view(v.shape)


class NormOut(NamedTuple):
    """rms_norm's outputs; None for those not asked for."""
    y: Optional[torch.Tensor]
    total: Optional[torch.Tensor]
    fp8: Optional[FP8Rows]


def _need(ok, msg):
    if not ok:
        raise ValueError(msg)


def _rows(t, name, K=None, rows=None, dtypes=(torch.bfloat16, torch.float16)):
    """A 2-D tensor whose rows are 16-byte aligned and contiguous."""
    if not (isinstance(t, torch.Tensor) and t.dtype in dtypes and t.dim() == 2 and
            (K is None or t.shape[1] == K) and (rows is None or t.shape[0] == rows)):
        want = "/".join(str(d).replace("torch.", "") for d in dtypes)
        raise ValueError(f"{name} must be a {want} [{'rows' if rows is None else rows}, "
                         f"{'K' if K is None else K}] tensor")
    if t.shape[0] and t.shape[1]:
        ld = _ld(t)
        _need((t.stride(1) == 1 or t.shape[1] == 1) and ld >= t.shape[1] and
              ld * t.element_size() % 16 == 0 and t.data_ptr() % 16 == 0,
              f"{name}'s rows must be contiguous and start on 16-byte boundaries")


def _ld(t):
    return t.stride(0) if t.shape[0] > 1 else _up16(t)


def _up16(t):
    """The smallest aligned stride of a single row, whose own is arbitrary."""
    e = 16 // t.element_size()
    return -(-t.shape[1] // e) * e


def _span(t):
    """(first byte, one past the last) of a 2-D or 1-D tensor."""
    n = 1 + sum((s - 1) * st for s, st in zip(t.shape, t.stride()))
    return t.data_ptr(), t.data_ptr() + n * t.element_size()


def _check_apart(out, name, others, same_ok=False):
    """`out` shares no memory with `others`; with same_ok it may be one of them
    (address, stride and type alike).  Column ranges of one buffer are apart."""
    if out.numel() == 0:
        return
    a0, a1 = _span(out)
    for t in others:
        if t is None or t.numel() == 0:
            continue
        b0, b1 = _span(t)
        if a1 <= b0 or b1 <= a0:
            continue
        if same_ok and b0 == a0 and t.dtype == out.dtype and \
                t.shape == out.shape and (t.shape[0] == 1 or t.stride(0) == out.stride(0)):
            continue
        if t.dim() == 2 and out.dim() == 2:
            pitch = out.stride(0) * out.element_size()
            if pitch == t.stride(0) * t.element_size() and pitch > 0:
                at = (b0 - a0) % pitch
                if out.shape[1] * out.element_size() <= at and \
                        at + t.shape[1] * t.element_size() <= pitch:
                    continue
        raise ValueError(f"{name} overlaps another tensor of the call")


class _Launch:
    """Device and stream of a call: checks that its tensors share a GPU, makes
    that device and `stream` current while outputs are allocated and work is
    queued, and marks tensors of another stream as used on this one."""

    __slots__ = ("stream", "handle", "_dev", "_ctx", "_tensors")

    def __init__(self, tensors, stream):
        dev = tensors[0].device
        _need(dev.type == "cuda", f"tensors must be on a GPU, not on {dev}")
        for t in tensors:
            if t is not None and t.device != dev:
                raise ValueError(f"tensors of one call must be on one device: {t.device} and {dev}")
        self._ctx = None
        if stream is None:
            self.handle = torch.cuda.current_stream(dev).cuda_stream
            if torch.cuda.current_device() != dev.index:
                self._ctx = torch.cuda.device(dev)
            return
        if isinstance(stream, int):
            stream = torch.cuda.ExternalStream(stream, device=dev)
        _need(stream.device == dev, f"stream is on {stream.device}, the tensors on {dev}")
        self.handle = stream.cuda_stream
        self._ctx = torch.cuda.stream(stream)          # makes its device current, too
        if stream != torch.cuda.current_stream(dev):
            for t in tensors:
                if t is not None:
                    t.record_stream(stream)

    def __enter__(self):
        if self._ctx is not None:
            self._ctx.__enter__()
        return self

    def __exit__(self, *exc):
        if self._ctx is not None:
            self._ctx.__exit__(*exc)


def _fp8_out(rows, K, scales, dev):
    codes = torch.empty((rows, K), dtype=torch.uint8, device=dev)
    if scales == "row":
        return FP8Rows(codes, torch.empty(rows, dtype=torch.float32, device=dev))
    return FP8Rows(codes, torch.empty((rows, K // 32), dtype=torch.uint8, device=dev))


def _check_scales(scales, K):
    _need(isinstance(scales, str) and scales in _FP8, 'scales must be "row" or "mx"')
    _need(scales != "mx" or K % 32 == 0, f'"mx" scales need a multiple of 32 columns, not {K}')


def rms_norm(x: torch.Tensor, weight: Optional[torch.Tensor] = None, *,
             residual: Optional[torch.Tensor] = None, eps: float = 1e-6,
             weight_offset: float = 0.0, want_y: bool = True, scales: Optional[str] = None,
             out: Optional[torch.Tensor] = None, total_out: Optional[torch.Tensor] = None,
             stream=None) -> NormOut:
    """s = x + residual (rounded to x's type; x alone without a residual), then
    s / sqrt(mean(s^2) + eps) * (weight_offset + weight): nvfp4_rmsnorm.

    x, residual [rows, K] bf16 or fp16 with K a multiple of 8, at most 32768;
    weight [K] of x's type (the factor is 1 without it).  Returns NormOut(y,
    total, fp8): y of x's type (want_y, or into `out`); total = s, given with a
    residual (into `total_out`, which like `out` may be x or residual); fp8 the
    8-bit rows when `scales` is "row" or "mx", rounded from the fp32 values."""
    _rows(x, "x")
    T, K = x.shape
    _need(8 <= K <= 32768 and K % 8 == 0, f"K must be a multiple of 8 in [8, 32768], not {K}")
    if residual is not None:
        _rows(residual, "residual", K, T, (x.dtype,))
    if weight is not None:
        _need(isinstance(weight, torch.Tensor) and weight.dtype == x.dtype and
              tuple(weight.shape) == (K,) and weight.is_contiguous() and
              weight.data_ptr() % 16 == 0,
              f"weight must be a contiguous 16-byte aligned {x.dtype} [{K}] tensor")
    if scales is not None:
        _check_scales(scales, K)
    _need(want_y or out is None, "out needs want_y")
    _need(residual is not None or total_out is None, "total_out needs a residual")
    _need(want_y or scales is not None or residual is not None,
          "nothing is asked for: want_y, scales or a residual")
    eps, weight_offset = float(eps), float(weight_offset)
    _need(0.0 <= eps < 3.4e38 and abs(weight_offset) < 3.4e38,
          "eps must be finite and >= 0, weight_offset finite")
    given = [x, residual, weight, out, total_out]
    if out is not None:
        _rows(out, "out", K, T, (x.dtype,))
        _check_apart(out, "out", (weight, total_out))
        _check_apart(out, "out", (x, residual), True)
    if total_out is not None:
        _rows(total_out, "total_out", K, T, (x.dtype,))
        _check_apart(total_out, "total_out", (weight,))
        _check_apart(total_out, "total_out", (x, residual), True)
    with _Launch(given, stream) as on:
        y = (torch.empty((T, K), dtype=x.dtype, device=x.device) if out is None else out) \
            if want_y else None
        total = None
        if residual is not None:
            total = torch.empty((T, K), dtype=x.dtype, device=x.device) \
                if total_out is None else total_out
        fp8 = None if scales is None else _fp8_out(T, K, scales, x.device)
        _lib.rmsnorm(_TYPES[x.dtype], x, _ld(x), residual, 0 if residual is None else _ld(residual),
                     weight, weight_offset, eps, T, K, total, 0 if total is None else _ld(total),
                     y, 0 if y is None else _ld(y), _lib.FP8_NONE if fp8 is None else _FP8[scales],
                     None if fp8 is None else fp8.codes, None if fp8 is None else fp8.scales,
                     on.handle)
    return NormOut(y, total, fp8)


def quantize_fp8(x: torch.Tensor, scales: str = "mx", *, stream=None) -> FP8Rows:
    """bf16 or fp16 rows [rows, K] -> FP8Rows with one fp32 scale per row
    ("row", K a multiple of 8) or one power-of-two scale per 32 elements ("mx",
    a multiple of 32): nvfp4_quantize_rows_fp8.  K is at most 32768."""
    _rows(x, "x")
    T, K = x.shape
    _need(8 <= K <= 32768 and K % 8 == 0, f"K must be a multiple of 8 in [8, 32768], not {K}")
    _check_scales(scales, K)
    with _Launch([x], stream) as on:
        fp8 = _fp8_out(T, K, scales, x.device)
        _lib.quantize_rows_fp8(_TYPES[x.dtype], x, _ld(x), T, K, _FP8[scales], fp8.codes,
                               fp8.scales, on.handle)
    return fp8


Operand = Union[torch.Tensor, FP8Rows]


def _operand(v, name):
    """(type, values, scales) of a linear operand, checked."""
    if isinstance(v, torch.Tensor):
        _rows(v, name)
        step, kind, scales = 8, _TYPES[v.dtype], None
    else:
        _need(isinstance(v, tuple) and len(v) == 2,
              f"{name} must be a bf16 or fp16 tensor or an FP8Rows")
        v, scales = v
        _rows(v, f"{name}.codes", dtypes=(torch.uint8,))
        _need(isinstance(scales, torch.Tensor) and scales.is_contiguous(),
              f"{name}.scales must be a contiguous tensor")
        if scales.dtype == torch.float32:
            step, kind, shape = 16, _lib.TYPE_FP8_ROW, (v.shape[0],)
        else:
            step, kind, shape = 32, _lib.TYPE_FP8_MX, (v.shape[0], v.shape[1] // 32)
            _need(scales.dtype == torch.uint8, f"{name}.scales must be fp32 or uint8")
        _need(tuple(scales.shape) == shape, f"{name}.scales must be of shape {shape}")
    K = v.shape[1]
    _need(K >= step and K % step == 0, f"{name} must have a multiple of {step} columns, not {K}")
    return kind, v, scales


def _plain(t, name, shape, dtypes=tuple(_TYPES)):
    """A tensor of `shape` with contiguous rows, without alignment beyond its type's."""
    _need(isinstance(t, torch.Tensor) and t.dtype in dtypes and tuple(t.shape) == shape and
          (t.numel() == 0 or ((t.stride(-1) == 1 or t.shape[-1] == 1) and
                              (t.dim() == 1 or t.shape[0] == 1 or t.stride(0) >= t.shape[1]))),
          f"{name} must be a {'/'.join(str(d).replace('torch.', '') for d in dtypes)} "
          f"{list(shape)} tensor with contiguous rows")


def linear(a: Operand, w: Operand, *, bias: Optional[torch.Tensor] = None,
           act: Optional[str] = None, gated: bool = False,
           residual: Optional[torch.Tensor] = None,
           out_dtype: Union[torch.dtype, str, None] = None,
           out: Optional[torch.Tensor] = None, stream=None) -> Operand:
    """act(a . w^T + bias) + residual, or with `gated` act(gate) * up + residual
    where w (and bias) hold N gate rows, then N up rows: nvfp4_linear.

    a [M, K] and w [N or 2N, K]: both bf16, both fp16, or both FP8Rows with the
    same kind of scales; K a multiple of 8 (16 for "row", 32 for "mx" operands).
    act: None, "silu", "gelu", "gelu_tanh" or "relu".  bias [N or 2N] and
    residual [M, N]: bf16, fp16 or fp32.  Returns [M, N] of `out_dtype` (a's
    type by default, bf16 for FP8Rows), or FP8Rows with "mx" scales for
    out_dtype "mx" (N a multiple of 32).  `out` receives the result and may be
    the residual itself."""
    kind, av, a_sc = _operand(a, "a")
    wkind, wv, w_sc = _operand(w, "w")
    _need(kind == wkind, "a and w must be of one type, with one kind of scales")
    M, K = av.shape
    _need(wv.shape[1] == K, f"w must have {K} columns, as a")
    _need(isinstance(gated, bool), "gated must be True or False")
    rows = wv.shape[0]
    _need(not gated or rows % 2 == 0, "a gated w has an even number of rows")
    N = rows // 2 if gated else rows
    try:
        act_id = _ACTS[act]
    except (KeyError, TypeError):
        raise ValueError(f"act must be one of {[k for k in _ACTS]}, not {act!r}") from None
    if bias is not None:
        _plain(bias, "bias", (rows,))
    if residual is not None:
        _plain(residual, "residual", (M, N))
    mx = isinstance(out_dtype, str)
    if mx:
        _need(out_dtype == "mx", f'out_dtype must be bf16, fp16, fp32 or "mx", not {out_dtype!r}')
        _need(N % 32 == 0, f'an "mx" result needs a multiple of 32 columns, not {N}')
        _need(out is None, 'out is not taken with out_dtype "mx"')
    else:
        if out_dtype is None:
            out_dtype = out.dtype if isinstance(out, torch.Tensor) else \
                torch.bfloat16 if a_sc is not None else av.dtype
        _need(out_dtype in _TYPES, f'out_dtype must be bf16, fp16, fp32 or "mx", not {out_dtype}')
        if out is not None:
            _plain(out, "out", (M, N), (out_dtype,))
            _check_apart(out, "out", (av, wv, a_sc, w_sc, bias))
            _check_apart(out, "out", (residual,), True)
    with _Launch([av, wv, a_sc, w_sc, bias, residual, out], stream) as on:
        dev = av.device
        out_scales = None
        if mx:
            res, out_scales = _fp8_out(M, N, "mx", dev)
        else:
            res = torch.empty((M, N), dtype=out_dtype, device=dev) if out is None else out
        p = _lib.Linear(
            av.data_ptr(), None if a_sc is None else a_sc.data_ptr(), wv.data_ptr(),
            None if w_sc is None else w_sc.data_ptr(), None if bias is None else bias.data_ptr(),
            None if residual is None else residual.data_ptr(), res.data_ptr(),
            None if out_scales is None else out_scales.data_ptr(),
            _ld(av), _ld(wv), 0 if residual is None else max(residual.stride(0), N),
            max(res.stride(0), N), M, N, K,
            kind, 0 if bias is None else _TYPES[bias.dtype],
            0 if residual is None else _TYPES[residual.dtype],
            _lib.TYPE_FP8_MX if mx else _TYPES[out_dtype], act_id, int(gated))
        n = _lib.linear_workspace_size(p)
        ws = torch.empty(n, dtype=torch.uint8, device=dev) if n else None
        _lib.linear(p, ws, n, on.handle)
    return FP8Rows(res, out_scales) if mx else res
