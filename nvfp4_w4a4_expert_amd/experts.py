"""The routed experts one operator at a time, on torch tensors.

``moe`` runs a layer's experts in 4 bits as one call.  These are its steps for
experts that are held in 16 or 8 bits:

    r = route(logits, k)                                   # ids, weights
    g = permute(r.ids, num_experts)                        # rows grouped by expert
    y = combine(rows_by_expert, r.weights, g.inv_pair, residual=h)

Conventions (ValueError for what does not fit, streams, memory, graphs, no
gradients) are those of ``dense``.
"""
from __future__ import annotations

from typing import NamedTuple, Optional

import torch

from . import _lib
from .dense import _FLOATS, _TYPES, _check_apart, _empty, _empty_strided, _need, _on, _rows


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
    if not (isinstance(t, torch.Tensor) and t.dtype == dtype and t.layout is torch.strided and
            tuple(t.shape) in shape and t.is_contiguous()):
        raise ValueError(f"{name} must be a contiguous {str(dtype).replace('torch.', '')} "
                         f"{' or '.join(str(list(s)) for s in shape)} tensor")
    return t.data_ptr()


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
