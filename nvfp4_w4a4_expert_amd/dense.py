"""The dense operators around the routed experts, on torch tensors.

``rms_norm`` adds the residual, normalises and quantises in one pass,
``block_norm`` does so behind a block's own last norm and gate, ``quantize_fp8``
makes the same 8-bit form of given rows, ``linear`` is a matrix product with
bias, activation (plain or gated) and residual in its epilogue, on bf16, fp16
or 8-bit operands, or with weights in 4 bits (``quantize_fp4``).  A dense
feed-forward beside the experts, in 8 bits end to end:

    n = rms_norm(x, weight, residual=h, scales="mx")       # n.y: the experts' bf16 input
    logits = linear(n.y, w_router, out_dtype=torch.float32)
    a = linear(n.fp8, w_gate_up, act="gelu_tanh", gated=True, out_dtype="mx")
    out = linear(a, w_down, residual=n.total)

All functions raise ValueError for tensors of the wrong dtype, shape, layout
or device, queue their work on `stream` (torch's current stream of the
tensors' device when None; an integer is a raw HIP stream handle, 0 the default
stream) and return without waiting.  A `stream` that is not the current one
neither waits for the work that makes the inputs, nor does later work of the
current stream wait for it: the caller orders them, and marks results that
other streams use (torch.Tensor.record_stream), since they are allocated on it.
All memory comes through torch, so calls can be captured into a graph.  Sizes
past the library's limits (2^31 rows or more; linear: rows longer than 8 MiB, a
result of more than 2^36 elements) raise NVFP4Error.  Forward only: no gradients
are recorded.
"""
from __future__ import annotations

import contextlib
import functools
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
    [rows] ("row") or UE8M0 uint8 [rows, K/32] ("mx"); experts' weights with the
    experts first in both.  Where an FP8Rows is taken, any (codes, scales) pair is."""
    codes: torch.Tensor
    scales: torch.Tensor

    def dequantize(self) -> torch.Tensor:
        """The values, in fp32 (with torch operations)."""
        v = self.codes.view(torch.float8_e4m3fn).float()
        if self.scales.dtype == torch.float32:
            return v * self.scales[..., None]
        s = self.scales.view(torch.float8_e8m0fnu).float()
        return (v.view(*s.shape, 32) * s[..., None]).view(v.shape)


class FP4Rows(NamedTuple):
    """Weights held in 4 bits: E2M1 codes uint8 [rows, K/2] (element 2j in the low
    nibble of byte j), block scales uint8 [rows, K/16] in E4M3 ("nv") or [rows,
    K/32] in UE8M0 ("mx"), and an fp32 tensor of one element that multiplies all
    of them, or None for 1."""
    codes: torch.Tensor
    scales: torch.Tensor
    scale: Optional[torch.Tensor] = None

    def dequantize(self) -> torch.Tensor:
        """The values, in fp32 (with torch operations)."""
        table = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device=self.codes.device)
        c = torch.stack([self.codes & 15, self.codes >> 4], 2).flatten(1).int()
        v = torch.where(c >= 8, -table[c & 7], table[c & 7])
        mx = self.codes.shape[1] * 2 == self.scales.shape[1] * 32
        s = self.scales.view(torch.float8_e8m0fnu if mx else torch.float8_e4m3fn).float()
        v = (v.view(*s.shape, 32 if mx else 16) * s[..., None]).view(v.shape)
        return v if self.scale is None else v * self.scale.reshape(())


class NormOut(NamedTuple):
    """rms_norm's outputs; None for those not asked for."""
    y: Optional[torch.Tensor]
    total: Optional[torch.Tensor]
    fp8: Optional[FP8Rows]


_HALF = (torch.bfloat16, torch.float16)
_BYTES = (torch.uint8,)
_FLOATS = tuple(_TYPES)


def _need(ok, msg):
    if not ok:
        raise ValueError(msg)


def _rows(t, name, K=None, rows=None, dtypes=_HALF):
    """(rows, K, row stride, address) of a 2-D tensor whose rows are contiguous
    and start on 16-byte boundaries (the stride of one row, which is arbitrary,
    as if it were followed by another)."""
    shape = t.shape if isinstance(t, torch.Tensor) and t.dtype in dtypes else ()
    if len(shape) != 2 or (K is not None and shape[1] != K) or (rows is not None and shape[0] != rows):
        want = "/".join(str(d).replace("torch.", "") for d in dtypes)
        raise ValueError(f"{name} must be a {want} [{'rows' if rows is None else rows}, "
                         f"{'K' if K is None else K}] tensor")
    T, K = shape
    if T > 0x7FFFFFFF or K > 0x7FFFFFFF:                       # (before outputs are allocated)
        _lib._check_size(T, f"rows of {name}")
        _lib._check_size(K, f"columns of {name}")
    per16 = 16 // t.element_size()
    ld, step = t.stride()
    if T <= 1:
        ld = -(-K // per16) * per16
    # (the strides first: those of a sparse tensor are 0, and it has no address)
    if (ld < K or ld % per16 or (step != 1 and K != 1) or t.data_ptr() % 16) and T and K:
        raise ValueError(f"{name}'s rows must be contiguous and start on 16-byte boundaries")
    return T, K, ld, t.data_ptr()


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


_HERE = contextlib.nullcontext()

# A small call costs the host more than the GPU (about 10 us against 3), so what
# every call does goes the short way: the current stream's handle, the current
# device and new tensors by torch's own C functions (0.1, 0.1 and 0.8 us where
# current_stream().cuda_stream, current_device() and new_empty take 1.9, 0.3 and
# 1.5), and no message is formed unless it is raised.
_raw_stream = torch._C._cuda_getCurrentRawStream if hasattr(torch._C, "_cuda_getCurrentRawStream") \
    else lambda index: torch.cuda.current_stream(index).cuda_stream
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
try:
    _empty_strided = torch._C._dynamo.guards._empty_strided_cuda       # on the current device
except AttributeError:
    def _empty_strided(shape, strides, dtype):
        return torch.empty_strided(shape, strides, dtype=dtype, device="cuda")


def _empty(rows, cols, dtype):
    return _empty_strided((rows, cols), (cols, 1), dtype)


def _on(tensors, stream):
    """(stream handle, context) of a call: checks that its tensors share a GPU;
    inside the context that device and `stream` are current, so outputs are
    allocated there.  Tensors of another stream are marked as used on this one."""
    index = tensors[0].get_device()
    for t in tensors:
        if t is not None and t.get_device() != index:
            raise ValueError(f"tensors of one call must be on one device: {t.device} and {tensors[0].device}")
    if index < 0 or not tensors[0].is_cuda:
        raise ValueError(f"tensors must be on a GPU, not on {tensors[0].device}")
    if stream is None:
        return _raw_stream(index), _HERE if _current_device() == index else torch.cuda.device(index)
    dev = tensors[0].device
    if isinstance(stream, int):                                # (ExternalStream takes 0 for a new stream)
        stream = torch.cuda.ExternalStream(stream, device=dev) if stream else torch.cuda.default_stream(dev)
    _need(isinstance(stream, torch.cuda.Stream), "stream must be a torch stream or a raw handle")
    _need(stream.device == dev, f"stream is on {stream.device}, the tensors on {dev}")
    if stream != torch.cuda.current_stream(dev):
        for t in tensors:
            if t is not None:
                t.record_stream(stream)
    return stream.cuda_stream, torch.cuda.stream(stream)       # makes its device current, too


def _fp8_out(rows, K, scales):
    codes = _empty(rows, K, torch.uint8)
    if scales == "row":
        return FP8Rows(codes, _empty_strided((rows,), (1,), torch.float32))
    return FP8Rows(codes, _empty(rows, K // 32, torch.uint8))


def _check_K(K):
    if not (8 <= K <= 32768 and K % 8 == 0):
        raise ValueError(f"K must be a multiple of 8 in [8, 32768], not {K}")


def _check_scales(scales, K):
    if not (isinstance(scales, str) and scales in _FP8):
        raise ValueError('scales must be "row" or "mx"')
    if scales == "mx" and K % 32:
        raise ValueError(f'"mx" scales need a multiple of 32 columns, not {K}')


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
    T, K, ldx, x_at = _rows(x, "x")
    _check_K(K)
    dtype = x.dtype
    r_at = w_at = y_at = total_at = codes_at = scales_at = None
    ldr = lds = 0
    ldy = K
    if residual is not None:
        _, _, ldr, r_at = _rows(residual, "residual", K, T, (dtype,))
    elif total_out is not None:
        raise ValueError("total_out needs a residual")
    elif not want_y and scales is None:
        raise ValueError("nothing is asked for: want_y, scales or a residual")
    if weight is not None:
        if not (isinstance(weight, torch.Tensor) and weight.dtype == dtype and
                weight.shape == (K,) and weight.is_contiguous() and weight.data_ptr() % 16 == 0):
            raise ValueError(f"weight must be a contiguous 16-byte aligned {dtype} [{K}] tensor")
        w_at = weight.data_ptr()
    if scales is not None:
        _check_scales(scales, K)
    eps, weight_offset = float(eps), float(weight_offset)
    if not (0.0 <= eps < 3.4e38 and -3.4e38 < weight_offset < 3.4e38):
        raise ValueError("eps must be finite and >= 0, weight_offset finite")
    if out is not None:
        _need(want_y, "out needs want_y")
        _, _, ldy, y_at = _rows(out, "out", K, T, (dtype,))
        _check_apart(out, "out", (weight, total_out))
        _check_apart(out, "out", (x, residual), True)
    if total_out is not None:
        _, _, lds, total_at = _rows(total_out, "total_out", K, T, (dtype,))
        _check_apart(total_out, "total_out", (weight,))
        _check_apart(total_out, "total_out", (x, residual), True)
    handle, ctx = _on((x, residual, weight, out, total_out), stream)
    with ctx:
        fp8, kind = None, _lib.FP8_NONE
        if want_y and out is None:
            out = _empty(T, K, dtype)
            y_at = out.data_ptr()
        if residual is not None and total_out is None:
            total_out, lds = _empty(T, K, dtype), K
            total_at = total_out.data_ptr()
        if scales is not None:
            kind = _FP8[scales]
            fp8 = _fp8_out(T, K, scales)
            codes_at, scales_at = fp8.codes.data_ptr(), fp8.scales.data_ptr()
        _lib.rmsnorm(_TYPES[dtype], x_at, ldx, r_at, ldr, w_at, weight_offset, eps, T, K,
                     total_at, lds, y_at, ldy, kind, codes_at, scales_at, handle)
    return NormOut(out, total_out, fp8)


_GATE_ACTS = {None: _lib.GATE_PLAIN, "none": _lib.GATE_PLAIN, "sigmoid": _lib.GATE_SIGMOID,
              "tanh": _lib.GATE_TANH}


def _gate(gate, T, K, dtype):
    """(address, row stride, columns, type) of a gate tensor that broadcasts to [T, K]."""
    shape = gate.shape
    n = len(shape)
    cols = shape[-1] if n else 0
    if not (gate.layout is torch.strided and (gate.dtype is dtype or gate.dtype is torch.float32) and
            (cols == 1 or cols == K) and (n == 1 or (n == 2 and shape[0] in (1, T)))):
        raise ValueError(f"gate must be a number or a {dtype} or fp32 tensor of [1], [{K}], [1, {K}], "
                         f"[{T}, 1] or [{T}, {K}]")
    ld = gate.stride(0) if n == 2 and shape[0] == T and T > 1 else 0
    at = gate.data_ptr()
    if cols == K and T and (gate.stride(-1) != 1 or at % 16 or ld * gate.element_size() % 16 or 0 < ld < K):
        raise ValueError("gate's rows must be contiguous and start on 16-byte boundaries")
    return at, ld, cols, _TYPES[gate.dtype]


def _weight(w, name, K, dtype):
    """The address of a norm's weight (0 without one), checked."""
    if w is None:
        return 0
    if isinstance(w, torch.Tensor) and w.dtype is dtype and w.shape == (K,) and w.is_contiguous():
        at = w.data_ptr()
        if not at % 16:
            return at
    raise ValueError(f"{name} must be a contiguous 16-byte aligned {dtype} [{K}] tensor")


def block_norm(x: torch.Tensor, residual: torch.Tensor, *, post_norm: bool = True,
               post_weight: Optional[torch.Tensor] = None,
               gate: Union[torch.Tensor, float, None] = None, gate_act: Optional[str] = None,
               residual_scale: float = 1.0, weight: Optional[torch.Tensor] = None,
               eps: float = 1e-6, weight_offset: float = 0.0, want_y: bool = True,
               scales: Optional[str] = None, out: Optional[torch.Tensor] = None,
               total_out: Optional[torch.Tensor] = None, stream=None) -> NormOut:
    """A block's end and the next one's start in one pass: nvfp4_block_norm.

        b = x / sqrt(mean(x^2) + eps) * (weight_offset + post_weight)   (x without post_norm)
        total = residual_scale * residual + gate * b                    (rounded to x's type)
        y = total / sqrt(mean(total^2) + eps) * (weight_offset + weight)

    x (the block's output) and residual [rows, K] bf16 or fp16 with K a multiple
    of 8, at most 32768; both weights [K] of x's type (the factor is 1 without).
    gate: a number, or a tensor of x's type or fp32, one element per row
    ([rows, 1]), per column ([K] or [1, K]), per element ([rows, K]) or one for
    all ([1]), through gate_act: None, "sigmoid" or "tanh" (tensors only).
    Returns NormOut(y, total, fp8) as rms_norm does, total always (into
    `total_out`, which like `out` may be x or residual); without want_y and
    scales only the total is computed."""
    T, K, ldx, x_at = _rows(x, "x")
    _check_K(K)
    dtype = x.dtype
    _, _, ldr, r_at = _rows(residual, "residual", K, T, (dtype,))
    if not (post_norm is True or post_norm is False):
        raise ValueError("post_norm must be True or False")
    if post_weight is not None and not post_norm:
        raise ValueError("post_weight needs post_norm")
    p_at, w_at = _weight(post_weight, "post_weight", K, dtype), _weight(weight, "weight", K, dtype)
    if weight is not None and not want_y and scales is None:
        raise ValueError("weight needs want_y or scales")
    try:
        act = _GATE_ACTS[gate_act]
    except (KeyError, TypeError):
        raise ValueError(f"gate_act must be one of {[k for k in _GATE_ACTS]}, not {gate_act!r}") from None
    g_at = ldg = gate_cols = gate_type = 0
    gate_scale = 1.0
    gate_t = gate if isinstance(gate, torch.Tensor) else None
    if gate_t is not None:
        g_at, ldg, gate_cols, gate_type = _gate(gate, T, K, dtype)
    elif act:
        raise ValueError("gate_act needs a gate tensor")
    elif gate is not None:
        try:
            gate_scale = float(gate)
        except (TypeError, ValueError):
            raise ValueError("gate must be a number or a tensor") from None
    if scales is not None:
        _check_scales(scales, K)
    eps, weight_offset, residual_scale = float(eps), float(weight_offset), float(residual_scale)
    if not (0.0 <= eps < 3.4e38 and -3.4e38 < weight_offset < 3.4e38 and
            -3.4e38 < gate_scale < 3.4e38 and -3.4e38 < residual_scale < 3.4e38):
        raise ValueError("eps must be finite and >= 0, weight_offset, gate and residual_scale finite")
    y_at = codes_at = scales_at = 0
    ldy = ldt = K
    if out is not None:
        _need(want_y, "out needs want_y")
        _, _, ldy, y_at = _rows(out, "out", K, T, (dtype,))
        _check_apart(out, "out", (post_weight, weight, gate_t, total_out))
        _check_apart(out, "out", (x, residual), True)
    if total_out is not None:
        _, _, ldt, t_at = _rows(total_out, "total_out", K, T, (dtype,))
        _check_apart(total_out, "total_out", (post_weight, weight, gate_t))
        _check_apart(total_out, "total_out", (x, residual), True)
    handle, ctx = _on((x, residual, post_weight, weight, gate_t, out, total_out), stream)
    with ctx:
        fp8, kind = None, _lib.FP8_NONE
        if want_y and out is None:
            out = _empty(T, K, dtype)
            y_at = out.data_ptr()
        if total_out is None:
            total_out = _empty(T, K, dtype)
            t_at = total_out.data_ptr()
        if scales is not None:
            kind = _FP8[scales]
            fp8 = _fp8_out(T, K, scales)
            codes_at, scales_at = fp8.codes.data_ptr(), fp8.scales.data_ptr()
        _lib.block_norm(_lib.pack_block_norm(
            x_at, r_at, p_at, w_at, g_at, t_at, y_at, codes_at, scales_at, ldx, ldr, ldg, ldt, ldy,
            T, K, _TYPES[dtype], post_norm, gate_type, gate_cols, act, kind,
            weight_offset, eps, gate_scale, residual_scale), handle)
    return NormOut(out, total_out, fp8)


def quantize_fp8(x: torch.Tensor, scales: str = "mx", *, stream=None) -> FP8Rows:
    """bf16 or fp16 rows [rows, K] -> FP8Rows with one fp32 scale per row
    ("row", K a multiple of 8) or one power-of-two scale per 32 elements ("mx",
    a multiple of 32): nvfp4_quantize_rows_fp8.  K is at most 32768."""
    T, K, ldx, x_at = _rows(x, "x")
    _check_K(K)
    _check_scales(scales, K)
    handle, ctx = _on((x,), stream)
    with ctx:
        fp8 = _fp8_out(T, K, scales)
        _lib.quantize_rows_fp8(_TYPES[x.dtype], x_at, ldx, T, K, _FP8[scales],
                               fp8.codes.data_ptr(), fp8.scales.data_ptr(), handle)
    return fp8


Operand = Union[torch.Tensor, FP8Rows]


def _operand(v, name):
    """(type, rows, K, row stride, address, values, scales, their address) of a
    linear operand, checked."""
    scales = scales_at = None
    if isinstance(v, torch.Tensor):
        rows, K, ld, at = _rows(v, name)
        step, kind = 8, _TYPES[v.dtype]
    else:
        if not (isinstance(v, tuple) and len(v) == 2):
            raise ValueError(f"{name} must be a bf16 or fp16 tensor or an FP8Rows")
        v, scales = v
        rows, K, ld, at = _rows(v, name, None, None, _BYTES)
        if not (isinstance(scales, torch.Tensor) and scales.is_contiguous()):
            raise ValueError(f"{name}'s scales must be a contiguous tensor")
        if scales.dtype == torch.float32:
            step, kind, shape = 16, _lib.TYPE_FP8_ROW, (rows,)
        else:
            step, kind, shape = 32, _lib.TYPE_FP8_MX, (rows, K // 32)
            _need(scales.dtype == torch.uint8, "block scales must be uint8, row scales fp32")
        if scales.shape != shape:
            raise ValueError(f"{name}'s scales must be of shape {shape}")
        scales_at = scales.data_ptr()
    if K < step or K % step:
        raise ValueError(f"{name} must have a multiple of {step} columns, not {K}")
    return kind, rows, K, ld, at, v, scales, scales_at


def _plain(t, name, shape, dtypes=_FLOATS):
    """The row stride of a tensor of `shape` with contiguous rows, aligned to its type."""
    if isinstance(t, torch.Tensor) and t.dtype in dtypes and t.shape == shape:
        st = t.stride()
        if len(shape) == 1:
            if st[0] == 1 or shape[0] <= 1:
                return 0
        else:
            ld = st[0] if shape[0] > 1 else shape[1]
            if ((st[1] == 1 or shape[1] == 1) and ld >= shape[1]) or 0 in shape:
                return max(ld, shape[1])
    raise ValueError(f"{name} must be a {'/'.join(str(d).replace('torch.', '') for d in dtypes)} "
                     f"{list(shape)} tensor with contiguous rows")


def quantize_fp4(w: torch.Tensor, scales: str = "nv", *, stream=None) -> FP4Rows:
    """bf16 weights [rows, K] -> FP4Rows, at load time: "nv" scales with the fp32
    scale max|w| / 2688 (1 for a matrix of zeros), or "mx" scales alone.  K is a
    multiple of 32.  The quantiser is the experts' own (nvfp4_quantize_experts and its
    UE8M0 form, the matrix as one expert).  Waits for the check that w is finite: the
    codes have no NaN or infinity."""
    T, K, ldw, _ = _rows(w, "w", None, None, (torch.bfloat16,))
    if not (isinstance(scales, str) and scales in ("nv", "mx")):
        raise ValueError('scales must be "nv" or "mx"')
    _need(K >= 32 and K % 32 == 0, f"w must have a multiple of 32 columns, not {K}")
    handle, ctx = _on((w,), stream)
    with ctx:
        _need(bool(torch.isfinite(w).all()), "w must be finite")
        nv = scales == "nv"
        codes, sf = _empty(T, K // 2, torch.uint8), _empty(T, K // (16 if nv else 32), torch.uint8)
        ends = torch.tensor([0, T], dtype=torch.int32, device=w.device)
        scale = gscale = None
        if nv:
            scale = _empty_strided((1,), (1,), torch.float32)
            _lib.expert_absmax(w, ldw, K, None, 1, ends, 1, T, scale, handle)
            top = scale.item() / 2688.0
            # (its reciprocal would leave fp32's range below 2^-126)
            scale.fill_(max(top, 2.0 ** -126) if top > 0 else 1.0)
            gscale = scale.reciprocal()
        quant = _lib.quantize_experts if nv else _lib.quantize_experts_mx
        quant(w, ldw, K, None, T, T, ends, 1, gscale, codes, sf, handle)
    return FP4Rows(codes, sf, scale)


def _fp4_operand(w, K):
    """(form, rows, row stride in bytes, codes, scales, gain or None) of FP4Rows
    weights against K columns, checked."""
    codes, scales, gain = w
    rows, half, ld, _ = _rows(codes, "w's codes", None, None, _BYTES)
    if half * 2 != K or K % 32:
        raise ValueError(f"w must have {K} columns, as a, a multiple of 32" if K % 32 == 0 else
                         f"a must have a multiple of 32 columns against FP4Rows, not {K}")
    if not (isinstance(scales, torch.Tensor) and scales.dtype == torch.uint8 and scales.layout is torch.strided and
            scales.is_contiguous() and scales.shape in ((rows, K // 16), (rows, K // 32))):
        raise ValueError(f"w's scales must be a contiguous uint8 tensor of shape [{rows}, {K // 16}] or [{rows}, {K // 32}]")
    mx = scales.shape[1] * 32 == K
    if not mx and scales.data_ptr() % 2:
        raise ValueError("w's scales must start on a 2-byte boundary")
    if gain is not None and not (isinstance(gain, torch.Tensor) and gain.dtype == torch.float32 and gain.numel() == 1 and
                                 gain.layout is torch.strided):
        raise ValueError("w's scale must be an fp32 tensor of one element, or None")
    return _lib.W4_MX if mx else _lib.W4_NV, rows, ld, codes, scales, gain


@functools.lru_cache(maxsize=4096)
def _workspace_bytes_w4(M, N, K, kind, out_type, gated, w4):
    return _lib.linear_w4_workspace_size(
        _lib.Linear(M=M, N=N, K=K, type=kind, out_type=out_type, gated=gated), w4)


@functools.lru_cache(maxsize=4096)
def _workspace_bytes(M, N, K, kind, out_type, gated):
    return _lib.linear_workspace_size(
        _lib.Linear(M=M, N=N, K=K, type=kind, out_type=out_type, gated=gated))


def linear(a: Operand, w: Union[Operand, FP4Rows], *, bias: Optional[torch.Tensor] = None,
           act: Optional[str] = None, gated: bool = False,
           residual: Optional[torch.Tensor] = None,
           out_dtype: Union[torch.dtype, str, None] = None,
           out: Optional[torch.Tensor] = None, stream=None) -> Operand:
    """act(a . w^T + bias) + residual, or with `gated` act(gate) * up + residual
    where w (and bias) hold N gate rows, then N up rows: nvfp4_linear.

    a [M, K] and w [N or 2N, K]: both bf16, both fp16, or both FP8Rows with the
    same kind of scales; K a multiple of 8 (16 for "row", 32 for "mx" operands).
    Or a in bf16 or fp16 and w as FP4Rows, K a multiple of 32 (nvfp4_linear_w4; all
    products exact, "mx" weights in bf16's range; for many rows w is written out
    in 16 bits, 2 * K bytes a row of memory for the call).
    act: None, "silu", "gelu", "gelu_tanh" or "relu".  bias [N or 2N] and
    residual [M, N]: bf16, fp16 or fp32.  Returns [M, N] of `out_dtype` (a's
    type by default, bf16 for FP8Rows), or FP8Rows with "mx" scales for
    out_dtype "mx" (N a multiple of 32).  `out` receives the result and may be
    the residual itself.

    FP8Rows with a 16-bit result and more than 16 rows may run on the scaled
    matrix instruction, which cuts each product to 2^-13 of the largest of its
    eight neighbours along K; every other form has exact products and fp32 sums.
    So a row may give other bits in a batch of 17 than in one of 16."""
    kind, M, K, lda, a_at, av, a_sc, a_sc_at = _operand(a, "a")
    fp4 = type(w) is FP4Rows
    gain = None
    if fp4:
        if a_sc is not None:
            raise ValueError("FP4Rows weights take a bf16 or fp16 a")
        w4, rows, ldw, wv, w_sc, gain = _fp4_operand(w, K)
        w_at, w_sc_at = wv.data_ptr(), w_sc.data_ptr()
    else:
        wkind, rows, wK, ldw, w_at, wv, w_sc, w_sc_at = _operand(w, "w")
        if kind != wkind:
            raise ValueError("a and w must be of one type, with one kind of scales")
        if wK != K:
            raise ValueError(f"w must have {K} columns, as a")
    if not (gated is False or gated is True):
        raise ValueError("gated must be True or False")
    if gated and rows % 2:
        raise ValueError("a gated w has an even number of rows")
    N = rows // 2 if gated else rows
    try:
        act_id = _ACTS[act]
    except (KeyError, TypeError):
        raise ValueError(f"act must be one of {[k for k in _ACTS]}, not {act!r}") from None
    bias_type = res_type = ldr = 0
    if bias is not None:
        _plain(bias, "bias", (rows,))
        bias_type = _TYPES[bias.dtype]
    if residual is not None:
        ldr = _plain(residual, "residual", (M, N))
        res_type = _TYPES[residual.dtype]
    mx = isinstance(out_dtype, str)
    ldo = N
    if mx:
        _need(out_dtype == "mx", 'out_dtype must be bf16, fp16, fp32 or "mx"')
        if N % 32:
            raise ValueError(f'an "mx" result needs a multiple of 32 columns, not {N}')
        _need(out is None, 'out is not taken with out_dtype "mx"')
        out_type = _lib.TYPE_FP8_MX
    else:
        if out_dtype is None:
            out_dtype = out.dtype if isinstance(out, torch.Tensor) else \
                torch.bfloat16 if a_sc is not None else av.dtype
        out_type = _TYPES.get(out_dtype)
        _need(out_type is not None, 'out_dtype must be bf16, fp16, fp32 or "mx"')
        if out is not None:
            ldo = _plain(out, "out", (M, N), (out_dtype,))
            _check_apart(out, "out", (av, wv, a_sc, w_sc, bias, gain))
            _check_apart(out, "out", (residual,), True)
    n = _workspace_bytes_w4(M, N, K, kind, out_type, gated, w4) if fp4 else \
        _workspace_bytes(M, N, K, kind, out_type, gated)      # NVFP4Error past the limits, before anything is allocated
    handle, ctx = _on((av, wv, a_sc, w_sc, bias, residual, out, gain), stream)
    with ctx:
        out_scales = None
        if mx:
            res, out_scales = _fp8_out(M, N, "mx")
        else:
            res = _empty(M, N, out_dtype) if out is None else out
        p = _lib.LinearFields(                               # (a's and w's sizes are checked)
            a_at, a_sc_at, w_at, w_sc_at, None if bias is None else bias.data_ptr(),
            None if residual is None else residual.data_ptr(), res.data_ptr(),
            None if out_scales is None else out_scales.data_ptr(), lda, ldw, ldr, ldo, M, N, K,
            kind, bias_type, res_type, out_type, act_id, gated)
        ws = _empty_strided((n,), (1,), torch.uint8) if n else None
        ws_at = None if ws is None else ws.data_ptr()
        if fp4:
            _lib.linear_w4(p, w4, None if gain is None else gain.data_ptr(), ws_at, n, handle)
        else:
            _lib.linear(p, ws_at, n, handle)
    return FP8Rows(res, out_scales) if mx else res
