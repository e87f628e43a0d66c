"""The routed experts one operator at a time, on torch tensors.

``moe`` runs a layer's experts in 4 bits as one call.  These are its steps for
experts that are held in 16 or 8 bits:

    r = route(logits, k)                                   # ids, weights
    g = permute(r.ids, num_experts)                        # rows grouped by expert
    h = grouped_linear(x, w13, g.offsets, index=g.src_pair, index_div=k, act="silu", gated=True)
    v = grouped_linear(h, w2, g.offsets, out_dtype=torch.float32)
    y = combine(v, r.weights, g.inv_pair, residual=x)

``ExpertsLayer`` holds a layer's weights and runs these.  Conventions (ValueError for what does not fit, streams, memory, graphs, no
gradients) are those of ``dense``.
"""
from __future__ import annotations

from typing import NamedTuple, Optional, Union

import torch

from . import _lib
from .dense import (_ACTS, _FLOATS, _HALF, _TYPES, FP8Rows, Operand, _check_apart, _empty, _empty_strided, _fp8_out, _need, _on,
                    _operand, _plain, _rows, quantize_fp8)


class Routing(NamedTuple):
    """route's outputs: int32 [tokens, k] and fp32 [tokens, k]."""
    ids: torch.Tensor
    weights: torch.Tensor


class Grouping(NamedTuple):
    """permute's outputs.  Pairs q = token * k + slot in the order of their
    experts: those of expert e are rows offsets[e] .. offsets[e + 1] (int32
    [experts + 1]); src_pair[row] = q and inv_pair[q] = row (int32 [pairs])."""
    offsets: torch.Tensor
    src_pair: torch.Tensor
    inv_pair: torch.Tensor


def _vector(t, name, dtype, shape):
    """The address of a contiguous tensor of one of the shapes, checked."""
    if isinstance(t, torch.Tensor) and t.dtype is dtype and t.layout is torch.strided and t.is_contiguous():
        have = t.shape
        for s in shape:
            if have == s:
                return t.data_ptr()
    raise ValueError(f"{name} must be a contiguous {str(dtype).replace('torch.', '')} "
                     f"{' or '.join(str(list(s)) for s in shape)} tensor")


def route(logits: torch.Tensor, k: int, *, stream=None) -> Routing:
    """The k largest of each token's fp32 logits [tokens, experts] (ties to the
    lower expert) and the softmax over them: nvfp4_route_topk.  At most 1024
    experts, k at most 32."""
    _need(isinstance(logits, torch.Tensor) and logits.dtype == torch.float32 and logits.dim() == 2 and
          logits.layout is torch.strided and logits.is_contiguous(),
          "logits must be a contiguous fp32 [tokens, experts] tensor")
    T, E = logits.shape
    _need(isinstance(k, int) and 1 <= k <= min(E, 32) and E <= 1024,
          f"k must be an integer in [1, {min(E, 32)}], the experts at most 1024")
    _lib._check_size(T, "rows of logits")
    handle, ctx = _on((logits,), stream)
    with ctx:
        out = Routing(_empty(T, k, torch.int32), _empty(T, k, torch.float32))
        _lib.route_topk(logits, T, E, k, out.ids, out.weights, handle)
    return out


def permute(ids: torch.Tensor, num_experts: int, *, stream=None) -> Grouping:
    """The pairs (token, slot) of int32 ids [tokens, k] grouped by expert, in
    order of (expert, token, slot): nvfp4_permute.  Pairs whose id is outside
    [0, num_experts) are left out: they have no row, their inv_pair and the last
    of src_pair are -1."""
    _need(isinstance(ids, torch.Tensor) and ids.dtype == torch.int32 and ids.dim() == 2 and
          ids.layout is torch.strided and ids.is_contiguous(), "ids must be a contiguous int32 [tokens, k] tensor")
    _need(isinstance(num_experts, int) and 1 <= num_experts <= 1024, "num_experts must be an integer in [1, 1024]")
    T, k = ids.shape
    _need(k >= 1, "ids must have a slot for each token at least")
    _lib._check_size(T * k, "pairs of ids")
    handle, ctx = _on((ids,), stream)
    with ctx:
        both = torch.full((2, T * k), -1, dtype=torch.int32, device=ids.device)
        out = Grouping(_empty_strided((num_experts + 1,), (1,), torch.int32), both[0], both[1])
        _lib.permute(ids, T, k, num_experts, *out, handle)
    return out


def _expert_weights(w, kind, like, name="w"):
    """(experts, rows, K, row stride, expert stride, values, scales) of a grouped
    product's weights, checked; kind is that of `like`, the operand beside them."""
    scales = None
    if kind in (_lib.TYPE_FP8_ROW, _lib.TYPE_FP8_MX):
        _need(isinstance(w, tuple) and len(w) == 2, f"{name} must be an FP8Rows, as {like}")
        w, scales = w
        dtype = torch.uint8
    else:
        dtype = torch.bfloat16 if kind == _lib.TYPE_BF16 else torch.float16
    _need(isinstance(w, torch.Tensor) and w.dtype == dtype and w.dim() == 3 and w.layout is torch.strided,
          f"{name} must be a {str(dtype).replace('torch.', '')} [experts, rows, K] tensor, as {like}")
    E, rows, K = w.shape
    _need(1 <= E <= 1024, f"{name} must hold between 1 and 1024 experts, not {E}")
    per16 = 16 // w.element_size()
    each, ld, step = w.stride()
    if rows <= 1:
        ld = -(-K // per16) * per16
    if E == 1:
        each = 0
    if rows and K and ((step != 1 and K != 1) or ld < K or ld % per16 or each % per16 or w.data_ptr() % 16 or
                       (E > 1 and each < (rows - 1) * ld + K)):
        raise ValueError(f"{name}'s rows must be contiguous, apart and start on 16-byte boundaries")
    if scales is not None:
        shape, dtype = ((E, rows), torch.float32) if kind == _lib.TYPE_FP8_ROW else ((E, rows, K // 32), torch.uint8)
        _vector(scales, f"{name}'s scales", dtype, (shape,))
    return E, rows, K, ld, each, w, scales


def grouped_linear(a: Operand, w: Operand, offsets: torch.Tensor, *, index: Optional[torch.Tensor] = None,
                   index_div: int = 1, bias: Optional[torch.Tensor] = None, act: Optional[str] = None,
                   gated: bool = False, out_dtype: Union[torch.dtype, str, None] = None,
                   out: Optional[torch.Tensor] = None, stream=None) -> Operand:
    """dense.linear for rows grouped by expert, each group with its own weight:
    nvfp4_grouped_linear.  Row m with offsets[e] <= m < offsets[e + 1] is

        act(a[row(m)] . w[e]^T + bias[e])     or     act(gate) * up

    with row(m) = m, or index[m] // index_div of an int32 `index` [rows] (with
    src_pair and k: each pair's token).  The groups' sizes stay on the device;
    rows behind the last group, or with an index outside a, are left as they
    were (in a new result: undefined).

    a [rows, K] bf16, fp16 or FP8Rows; w [experts, N or 2N, K] of its type, at
    most 1024 experts, or FP8Rows of codes [experts, N or 2N, K] with scales
    [experts, N or 2N] or [experts, N or 2N, K/32]; K as for linear.  offsets
    int32 [experts + 1]; bias [experts, N or 2N] bf16, fp16 or fp32.  Returns
    [rows, N] of `out_dtype` (a's type by default, bf16 for FP8Rows), or FP8Rows
    with "mx" scales for "mx" (N a multiple of 32).  `out` receives the result.
    Products are exact and sums fp32, of FP8Rows too."""
    kind, T, K, lda, a_at, av, a_sc, a_sc_at = _operand(a, "a")
    E, rows, wK, ldw, each, wv, w_sc = _expert_weights(w, kind, "a")
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
    offsets_at = _vector(offsets, "offsets", torch.int32, ((E + 1,),))
    P, index_at = T, 0
    if index is not None:
        _need(isinstance(index, torch.Tensor) and index.dim() == 1, "index must be an int32 [rows] tensor")
        P = index.shape[0]
        index_at = _vector(index, "index", torch.int32, ((P,),))
    if not (isinstance(index_div, int) and 1 <= index_div <= 0x7FFFFFFF):
        raise ValueError("index_div must be a positive integer")
    bias_type = bias_at = 0
    if bias is not None:
        _need(isinstance(bias, torch.Tensor) and bias.dtype in _FLOATS, "bias must be a bf16, fp16 or fp32 tensor")
        bias_at, bias_type = _vector(bias, "bias", bias.dtype, ((E, rows),)), _TYPES[bias.dtype]
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
            ldo = _plain(out, "out", (P, N), (out_dtype,))
            _check_apart(out, "out", (av, wv, a_sc, w_sc, bias, offsets, index))
    _lib._check_size(P, "rows of the result")
    _lib._check_size(rows, "rows of w")
    handle, ctx = _on((av, wv, a_sc, w_sc, bias, offsets, index, out), stream)
    with ctx:
        out_scales = None
        if mx:
            res, out_scales = _fp8_out(P, N, "mx")
        else:
            res = _empty(P, N, out_dtype) if out is None else out
        _lib.grouped_linear(_lib.pack_grouped_linear(
            a_at, a_sc_at or 0, wv.data_ptr(), 0 if w_sc is None else w_sc.data_ptr(), bias_at, offsets_at,
            index_at, res.data_ptr(), 0 if out_scales is None else out_scales.data_ptr(), lda, ldw, each,
            ldo, P, T, E, N, K, index_div, kind, bias_type, out_type, act_id, gated), handle)
    return FP8Rows(res, out_scales) if mx else res


def combine(values: torch.Tensor, weights: torch.Tensor, inv_pair: torch.Tensor, *,
            residual: Optional[torch.Tensor] = None, out_dtype: Optional[torch.dtype] = None,
            out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """out[t] = residual[t] + sum_j weights[t, j] * values[inv_pair[t * k + j]], the
    experts' rows back in token order: nvfp4_combine.

    values [rows, H] bf16, fp16 or fp32 with H a multiple of 8; weights fp32
    [tokens, k]; inv_pair int32 [tokens * k] or [tokens, k], pairs outside
    [0, rows) are left out; residual [tokens, H].  Returns [tokens, H] of
    `out_dtype` (bf16 by default); `out` receives it and may be the residual."""
    P, H, ldv, v_at = _rows(values, "values", None, None, _FLOATS)
    _need(8 <= H <= 1 << 24 and H % 8 == 0, f"values must have a multiple of 8 columns, at most 2^24, not {H}")
    _need(isinstance(weights, torch.Tensor) and weights.dim() == 2, "weights must be an fp32 [tokens, k] tensor")
    T, k = weights.shape
    _need(1 <= k <= 1024, f"k must be in [1, 1024], not {k}")
    w_at = _vector(weights, "weights", torch.float32, ((T, k),))
    inv_at = _vector(inv_pair, "inv_pair", torch.int32, ((T * k,), (T, k)))
    r_at, ldr, r_type = None, 0, 0
    if residual is not None:
        _, _, ldr, r_at = _rows(residual, "residual", H, T, _FLOATS)
        r_type = _TYPES[residual.dtype]
    if out_dtype is None:
        out_dtype = out.dtype if isinstance(out, torch.Tensor) else torch.bfloat16
    _need(out_dtype in _TYPES, "out_dtype must be bf16, fp16 or fp32")
    ldo = H
    if out is not None:
        _, _, ldo, _ = _rows(out, "out", H, T, (out_dtype,))
        _check_apart(out, "out", (values, weights, inv_pair.view(-1)))
        _check_apart(out, "out", (residual,), True)
    handle, ctx = _on((values, weights, inv_pair, residual, out), stream)
    with ctx:
        if out is None:
            out = _empty(T, H, out_dtype)
        _lib.combine(_TYPES[values.dtype], v_at, ldv, P, w_at, inv_at, T, k, H, r_type, r_at, ldr,
                     _TYPES[out_dtype], out.data_ptr(), ldo, handle)
    return out


class ExpertsLayer:
    """A layer's routed experts held in 16 or 8 bits: what moe.NVFP4MoELayer runs
    in 4.  w13 [experts, 2 * inter, hidden] (gate rows, then up rows) and w2
    [experts, hidden, inter]: bf16 or fp16 tensors, or FP8Rows (codes and scales
    with the experts first) of which `quantized` makes a layer.  act: the gate's
    activation; bias13 [experts, 2 * inter], bias2 [experts, hidden]."""

    def __init__(self, w13: Operand, w2: Operand, *, act: str = "silu", bias13: Optional[torch.Tensor] = None,
                 bias2: Optional[torch.Tensor] = None):
        if isinstance(w13, tuple) and len(w13) == 2 and isinstance(w13[1], torch.Tensor):
            kind, step = (_lib.TYPE_FP8_ROW, 16) if w13[1].dtype == torch.float32 else (_lib.TYPE_FP8_MX, 32)
        else:
            _need(isinstance(w13, torch.Tensor) and w13.dtype in _HALF, "w13 must be a bf16 or fp16 tensor or an FP8Rows")
            kind, step = _TYPES[w13.dtype], 8
        E, rows, H = _expert_weights(w13, kind, "w13", "w13")[:3]
        E2, H2, inter = _expert_weights(w2, kind, "w13", "w2")[:3]
        _need(rows == 2 * inter and E2 == E and H2 == H,
              f"w13 [{E}, {rows}, {H}] must be [experts, 2 * inter, hidden] and w2 [{E2}, {H2}, {inter}] [experts, hidden, inter]")
        _need(H >= step and inter >= step and H % step == 0 and inter % step == 0,
              f"hidden and inter must be multiples of {step}, not {H} and {inter}")
        for b, name, n in ((bias13, "bias13", rows), (bias2, "bias2", H)):
            if b is not None:
                _need(isinstance(b, torch.Tensor) and b.dtype in _FLOATS, f"{name} must be a bf16, fp16 or fp32 tensor")
                _vector(b, name, b.dtype, ((E, n),))
        _need(act is None or isinstance(act, str) and act in _ACTS, f"act must be one of {[k for k in _ACTS]}, not {act!r}")
        self.w13, self.w2, self.act, self.bias13, self.bias2 = w13, w2, act, bias13, bias2
        self.scales = {_lib.TYPE_FP8_ROW: "row", _lib.TYPE_FP8_MX: "mx"}.get(kind)
        self.num_experts = E

    @classmethod
    def quantized(cls, w13: torch.Tensor, w2: torch.Tensor, scales: str = "mx", **kw) -> "ExpertsLayer":
        """The layer in 8 bits, from bf16 or fp16 weights."""
        def fp8(w):
            _need(isinstance(w, torch.Tensor) and w.dim() == 3, "w13 and w2 must be [experts, rows, K] tensors")
            q = quantize_fp8(w.reshape(-1, w.shape[2]), scales)
            return FP8Rows(*(t.view(*w.shape[:2], *t.shape[1:]) for t in q))
        return cls(fp8(w13), fp8(w2), **kw)

    def forward(self, x: Operand, logits: torch.Tensor, k: int, residual: Optional[torch.Tensor] = None,
                out_dtype: Optional[torch.dtype] = None, stream=None) -> torch.Tensor:
        """x [tokens, hidden] and fp32 logits [tokens, experts] -> [tokens, hidden] of
        `out_dtype` (x's type by default, bf16 for FP8Rows).  A layer in 8 bits takes x as
        FP8Rows with its kind of scales, or quantises it.  The experts' rows stay in fp32
        up to the combine, as in moe."""
        rows = x[0] if isinstance(x, tuple) and x else x
        _need(isinstance(rows, torch.Tensor) and rows.dim() == 2, "x must be a [tokens, hidden] tensor or an FP8Rows")
        # (an index past x's rows would leave rows unwritten, an expert past the weights out)
        _need(isinstance(logits, torch.Tensor) and logits.shape == (rows.shape[0], self.num_experts),
              f"logits must be an fp32 [{rows.shape[0]}, {self.num_experts}] tensor")
        if out_dtype is None:
            out_dtype = x.dtype if isinstance(x, torch.Tensor) else torch.bfloat16
        if self.scales is not None and isinstance(x, torch.Tensor):
            x = quantize_fp8(x, self.scales, stream=stream)
        r = route(logits, k, stream=stream)
        g = permute(r.ids, self.num_experts, stream=stream)
        h = grouped_linear(x, self.w13, g.offsets, index=g.src_pair, index_div=k, bias=self.bias13, act=self.act,
                           gated=True, out_dtype="mx" if self.scales == "mx" else None, stream=stream)
        if self.scales == "row":
            h = quantize_fp8(h, "row", stream=stream)
        v = grouped_linear(h, self.w2, g.offsets, bias=self.bias2, out_dtype=torch.float32, stream=stream)
        return combine(v, r.weights, g.inv_pair, residual=residual, out_dtype=out_dtype, stream=stream)
