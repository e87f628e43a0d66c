"""ctypes binding of libnvfp4moe.so (include/nvfp4_moe.h).

Argument marshalling only: every function forwards to the C entry point of
the same name.  Device buffers are torch tensors on the GPU (their
``data_ptr()`` is passed); the stream is torch's current stream unless one
is given.  Errors come back as :class:`NVFP4Error`.

The library must have been built (``python -m nvfp4_w4a4_expert_amd.build``);
importing this module without it raises ImportError — there is no fallback.
"""
from __future__ import annotations

import ctypes
import os
import struct
from typing import Optional

import numpy as np

from .build import LIB_PATH

(OK, ERR_INVALID_ARG, ERR_BAD_SCALE, ERR_WORKSPACE, ERR_DEVICE, ERR_UNSUPPORTED,
 ERR_TOO_LARGE) = range(7)
NOALLOC_SCRATCH_BYTES = 64 << 20      # NVFP4_NOALLOC_SCRATCH_BYTES
SLOT_OK, SLOT_UNWRITTEN, SLOT_NAN, SLOT_INF, SLOT_NONPOSITIVE, SLOT_RECIP_OVERFLOW = range(6)

if not os.path.exists(LIB_PATH):
    raise ImportError(f"{LIB_PATH} is not built; run `python -m nvfp4_w4a4_expert_amd.build`")

_lib = ctypes.CDLL(LIB_PATH)

_p = ctypes.c_void_p
_i32 = ctypes.c_int32
_i64 = ctypes.c_int64


class MoEWeights(ctypes.Structure):
    _fields_ = [
        ("w13", _p), ("w13_sf", _p), ("w13_scale2", _p),
        ("w2", _p), ("w2_sf", _p), ("w2_scale2", _p),
        ("w13_input_scale", _p), ("w2_input_scale", _p),
        ("a1_gscale", _p), ("a2_gscale", _p),
        ("num_experts", _i32), ("hidden", _i32), ("inter", _i32),
    ]


class MoEDebug(ctypes.Structure):
    _fields_ = [
        ("topk_ids", _p), ("topk_weights", _p), ("expert_offsets", _p),
        ("src_pair", _p), ("inv_pair", _p), ("a1_codes", _p), ("a1_sf", _p),
        ("c1", _p), ("h", _p), ("a2_codes", _p), ("a2_sf", _p), ("c2", _p),
        ("stage_events", ctypes.POINTER(_p)),
    ]


class LinearFields(ctypes.Structure):
    """nvfp4_linear_t.  ctypes drops the upper bits of a size past 32 bits; Linear
    below refuses it."""
    _fields_ = [
        ("a", _p), ("a_scales", _p), ("w", _p), ("w_scales", _p),
        ("bias", _p), ("residual", _p), ("out", _p), ("out_scales", _p),
        ("lda", _i64), ("ldw", _i64), ("ldr", _i64), ("ldo", _i64),
        ("M", _i32), ("N", _i32), ("K", _i32),
        ("type", _i32), ("bias_type", _i32), ("residual_type", _i32), ("out_type", _i32),
        ("act", _i32), ("gated", _i32),
    ]


class Linear(LinearFields):
    """nvfp4_linear_t with sizes that fit its 32 bits, else NVFP4Error."""

    def __init__(self, *args, **fields):
        super().__init__(*args, **fields)
        for name, given in [*zip(_LINEAR_NAMES, args), *fields.items()]:
            if name in ("M", "N", "K"):
                _check_size(given, f"nvfp4_linear_t.{name}")


class BlockNorm(ctypes.Structure):
    """nvfp4_block_norm_t."""
    _fields_ = [
        ("x", _p), ("residual", _p), ("post_weight", _p), ("weight", _p), ("gate", _p),
        ("total_out", _p), ("y_out", _p), ("codes", _p), ("scales", _p),
        ("ldx", _i64), ("ldr", _i64), ("ldg", _i64), ("ldt", _i64), ("ldy", _i64),
        ("num_rows", _i32), ("K", _i32),
        ("type", _i32), ("post", _i32), ("gate_type", _i32), ("gate_cols", _i32),
        ("gate_act", _i32), ("fp8", _i32),
        ("weight_offset", ctypes.c_float), ("eps", ctypes.c_float),
        ("gate_scale", ctypes.c_float), ("residual_scale", ctypes.c_float),
    ]


class GroupedLinear(ctypes.Structure):
    """nvfp4_grouped_linear_t."""
    _fields_ = [
        ("a", _p), ("a_scales", _p), ("w", _p), ("w_scales", _p), ("bias", _p),
        ("offsets", _p), ("index", _p), ("out", _p), ("out_scales", _p),
        ("lda", _i64), ("ldw", _i64), ("w_each", _i64), ("ldo", _i64),
        ("num_rows", _i32), ("a_rows", _i32), ("num_experts", _i32), ("N", _i32), ("K", _i32),
        ("index_div", _i32), ("type", _i32), ("bias_type", _i32), ("out_type", _i32),
        ("act", _i32), ("gated", _i32),
    ]


# The same two as bytes: packing them takes a quarter of the time of a ctypes structure.
# Addresses are integers, 0 for NULL.
pack_block_norm = struct.Struct("9P5q8i4f").pack
pack_grouped_linear = struct.Struct("9P4q11i4x").pack


_LINEAR_NAMES = tuple(name for name, _ in LinearFields._fields_)

FP8_NONE = -1
TYPE_BF16, TYPE_FP16, TYPE_FP32, TYPE_FP8_ROW, TYPE_FP8_MX = range(5)
GATE_PLAIN, GATE_SIGMOID, GATE_TANH = range(3)
W4_NV, W4_MX = range(2)
ACT_NONE, ACT_SILU, ACT_GELU, ACT_GELU_TANH, ACT_RELU = range(5)

MOE_STAGES = ("route", "permute", "quantize_a1", "gemm1_w13", "gemm2_w2", "combine")


_SIGS = {
    "nvfp4_status_string": (ctypes.c_char_p, [_i32]),
    "nvfp4_abi_version": (_i32, []),
    "nvfp4_validate_scales": (_i32, [_p, _p, _i32, _p, _p, _p]),
    "nvfp4_quantize_experts": (_i32, [_p, _i64, _i32, _p, _i32, _i32, _p, _i32, _p, _p, _p, _p]),
    "nvfp4_quantize_pairs": (_i32, [_p, _i64, _i32, _i32, _i32, _p, _p, _i32, _p, _p, _p, _i32, _p]),
    "nvfp4_quantize_experts_fp16": (_i32, [_p, _i64, _i32, _p, _i32, _i32, _p, _i32, _p, _p, _p, _p]),
    "nvfp4_route_topk": (_i32, [_p, _i32, _i32, _i32, _p, _p, _p]),
    "nvfp4_permute": (_i32, [_p, _i32, _i32, _i32, _p, _p, _p, _p]),
    "nvfp4_expert_absmax": (_i32, [_p, _i64, _i32, _p, _i32, _p, _i32, _i32, _p, _p]),
    "nvfp4_calibrate_input_scales": (_i32, [_p, _i64, _i32, _p, _i32, _p, _i32, _i32, _p, _p, _p]),
    "nvfp4_selftest_conversions": (_i32, [_p, _p]),
    "nvfp4_moe_pack_weights": (_i32, [_i32, _p, _p, _i32, _i32, _i32, _p, _p, _p]),
    "nvfp4_moe_workspace_size": (_i32, [_i32, _i32, ctypes.POINTER(MoEWeights), ctypes.POINTER(ctypes.c_size_t)]),
    "nvfp4_moe_forward": (_i32, [ctypes.POINTER(MoEWeights), _p, _p, _i32, _i32, _p, _p, _p,
                                 ctypes.c_size_t, ctypes.POINTER(MoEDebug), _p]),
    "nvfp4_quantize_experts_mx": (_i32, [_p, _i64, _i32, _p, _i32, _i32, _p, _i32, _p, _p, _p, _p]),
    "nvfp4_quantize_pairs_mx": (_i32, [_p, _i64, _i32, _i32, _i32, _p, _p, _i32, _p, _p, _p, _i32, _p]),
    "nvfp4_moe_pack_weights_mx": (_i32, [_i32, _p, _p, _i32, _i32, _i32, _p, _p, _p]),
    "nvfp4_moe_forward_mx": (_i32, [ctypes.POINTER(MoEWeights), _p, _p, _i32, _i32, _p, _p, _p,
                                    ctypes.c_size_t, ctypes.POINTER(MoEDebug), _p]),
    "nvfp4_moe_workspace_size_w4a16": (_i32, [_i32, _i32, ctypes.POINTER(MoEWeights),
                                              ctypes.POINTER(ctypes.c_size_t)]),
    "nvfp4_moe_forward_w4a16": (_i32, [ctypes.POINTER(MoEWeights), _p, _p, _i32, _i32, _p, _p,
                                       _p, ctypes.c_size_t, ctypes.POINTER(MoEDebug), _p]),
    "nvfp4_moe_forward_noalloc": (_i32, [ctypes.POINTER(MoEWeights), _p, _p, _i32, _i32, _p, _p,
                                         ctypes.POINTER(MoEDebug), _p]),
    "nvfp4_rmsnorm": (_i32, [_i32, _p, _i64, _p, _i64, _p, ctypes.c_float, ctypes.c_float, _i32,
                             _i32, _p, _i64, _p, _i64, _i32, _p, _p, _p]),
    "nvfp4_block_norm": (_i32, [_p, _p]),
    "nvfp4_quantize_rows_fp8": (_i32, [_i32, _p, _i64, _i32, _i32, _i32, _p, _p, _p]),
    "nvfp4_linear_workspace_size": (_i32, [ctypes.POINTER(LinearFields), ctypes.POINTER(ctypes.c_size_t)]),
    "nvfp4_linear": (_i32, [ctypes.POINTER(LinearFields), _p, ctypes.c_size_t, _p]),
    "nvfp4_linear_w4_workspace_size": (_i32, [ctypes.POINTER(LinearFields), _i32, ctypes.POINTER(ctypes.c_size_t)]),
    "nvfp4_linear_w4": (_i32, [ctypes.POINTER(LinearFields), _i32, _p, _p, ctypes.c_size_t, _p]),
    "nvfp4_grouped_linear": (_i32, [_p, _p]),
    "nvfp4_combine": (_i32, [_i32, _p, _i64, _i32, _p, _p, _i32, _i32, _i32, _i32, _p, _i64, _i32,
                             _p, _i64, _p]),
}

EXPORTED = tuple(_SIGS)

for _name, (_res, _args) in _SIGS.items():
    _fn = getattr(_lib, _name)
    _fn.restype = _res
    _fn.argtypes = _args


class NVFP4Error(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {status_string(status)} (status {status})")


def status_string(status: int) -> str:
    return _lib.nvfp4_status_string(status).decode()


def abi_version() -> int:
    return int(_lib.nvfp4_abi_version())


def _check(status: int, where: str) -> None:
    if status != OK:
        raise NVFP4Error(status, where)


def _check_size(n: int, where: str) -> None:
    """The C entry points take sizes in 32 bits; ctypes would cut a longer one."""
    if not -0x80000000 <= n <= 0x7FFFFFFF:
        raise NVFP4Error(ERR_UNSUPPORTED, f"{where} = {n}")


def _ptr(t) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _stream(stream) -> Optional[int]:
    if stream is not None:
        return stream if isinstance(stream, int) else stream.cuda_stream
    import torch
    return torch.cuda.current_stream().cuda_stream


# --- host -------------------------------------------------------------------

def validate_scales(input_scale: np.ndarray, written: Optional[np.ndarray] = None):
    """Host arrays in; returns (status, gscale or None, slot_status, num_bad)."""
    x = np.ascontiguousarray(input_scale, dtype=np.float32)
    E = x.size
    wr = None if written is None else np.ascontiguousarray(written, dtype=np.uint8)
    gs = np.full(E, np.nan, dtype=np.float32)
    st = np.full(E, -1, dtype=np.int32)
    nb = ctypes.c_int32(-1)
    status = _lib.nvfp4_validate_scales(
        x.ctypes.data, None if wr is None else wr.ctypes.data, E, gs.ctypes.data,
        st.ctypes.data, ctypes.addressof(nb))
    return status, (gs if status == OK else None), st, nb.value


# --- device -----------------------------------------------------------------

def quantize_experts(x, ldx: int, K: int, src_row, num_src_rows: int, P: int, expert_offsets,
                     num_experts: int, gscale, codes, sf, stream=None):
    _check(_lib.nvfp4_quantize_experts(_ptr(x), ldx, K, _ptr(src_row), num_src_rows, P,
                                       _ptr(expert_offsets), num_experts, _ptr(gscale),
                                       _ptr(codes), _ptr(sf), _stream(stream)),
           "nvfp4_quantize_experts")


def quantize_experts_fp16(x, ldx: int, K: int, src_row, num_src_rows: int, P: int,
                          expert_offsets, num_experts: int, gscale, codes, sf, stream=None):
    _check(_lib.nvfp4_quantize_experts_fp16(_ptr(x), ldx, K, _ptr(src_row), num_src_rows, P,
                                            _ptr(expert_offsets), num_experts, _ptr(gscale),
                                            _ptr(codes), _ptr(sf), _stream(stream)),
           "nvfp4_quantize_experts_fp16")


def quantize_pairs(x, ldx: int, num_rows: int, K: int, topk: int, expert_idx, dst_row,
                   num_experts: int, gscale, codes, sf, num_dst_rows: int, stream=None):
    _check(_lib.nvfp4_quantize_pairs(_ptr(x), ldx, num_rows, K, topk, _ptr(expert_idx),
                                     _ptr(dst_row), num_experts, _ptr(gscale), _ptr(codes),
                                     _ptr(sf), num_dst_rows, _stream(stream)),
           "nvfp4_quantize_pairs")


def route_topk(logits, num_tokens: int, num_experts: int, k: int, ids, weights, stream=None):
    _check(_lib.nvfp4_route_topk(_ptr(logits), num_tokens, num_experts, k, _ptr(ids),
                                 _ptr(weights), _stream(stream)), "nvfp4_route_topk")


def permute(ids, num_tokens: int, k: int, num_experts: int, expert_offsets, src_pair, inv_pair,
            stream=None):
    _check(_lib.nvfp4_permute(_ptr(ids), num_tokens, k, num_experts, _ptr(expert_offsets),
                              _ptr(src_pair), _ptr(inv_pair), _stream(stream)), "nvfp4_permute")


def expert_absmax(x, ldx: int, K: int, src, src_div: int, expert_offsets, num_experts: int,
                  num_rows: int, amax_out, stream=None):
    _check(_lib.nvfp4_expert_absmax(_ptr(x), ldx, K, _ptr(src), src_div, _ptr(expert_offsets),
                                    num_experts, num_rows, _ptr(amax_out), _stream(stream)),
           "nvfp4_expert_absmax")


def calibrate_input_scales(x, ldx: int, K: int, src, src_div: int, expert_offsets,
                           num_experts: int, num_rows: int, input_scale_out, written_out,
                           stream=None):
    _check(_lib.nvfp4_calibrate_input_scales(_ptr(x), ldx, K, _ptr(src), src_div,
                                             _ptr(expert_offsets), num_experts, num_rows,
                                             _ptr(input_scale_out), _ptr(written_out),
                                             _stream(stream)),
           "nvfp4_calibrate_input_scales")


def selftest_conversions(mismatches, stream=None):
    _check(_lib.nvfp4_selftest_conversions(_ptr(mismatches), _stream(stream)),
           "nvfp4_selftest_conversions")


def moe_pack_weights(projection: int, codes, sf, num_experts: int, hidden: int, inter: int,
                     codes_out, sf_out, stream=None):
    _check(_lib.nvfp4_moe_pack_weights(projection, _ptr(codes), _ptr(sf), num_experts, hidden,
                                       inter, _ptr(codes_out), _ptr(sf_out), _stream(stream)),
           "nvfp4_moe_pack_weights")


def moe_workspace_size(num_tokens: int, k: int, weights: MoEWeights) -> int:
    n = ctypes.c_size_t(0)
    _check(_lib.nvfp4_moe_workspace_size(num_tokens, k, ctypes.byref(weights), ctypes.byref(n)),
           "nvfp4_moe_workspace_size")
    return int(n.value)


def moe_forward(weights: MoEWeights, x, router_logits, num_tokens: int, k: int, residual, out,
                workspace, workspace_bytes: int, debug: Optional[MoEDebug] = None, stream=None):
    _check(_lib.nvfp4_moe_forward(ctypes.byref(weights), _ptr(x), _ptr(router_logits),
                                  num_tokens, k, _ptr(residual), _ptr(out), _ptr(workspace),
                                  workspace_bytes, None if debug is None else ctypes.byref(debug),
                                  _stream(stream)), "nvfp4_moe_forward")


def moe_workspace_size_w4a16(num_tokens: int, k: int, weights: MoEWeights) -> int:
    n = ctypes.c_size_t(0)
    _check(_lib.nvfp4_moe_workspace_size_w4a16(num_tokens, k, ctypes.byref(weights),
                                               ctypes.byref(n)),
           "nvfp4_moe_workspace_size_w4a16")
    return int(n.value)


def moe_forward_w4a16(weights: MoEWeights, x, router_logits, num_tokens: int, k: int, residual,
                      out, workspace, workspace_bytes: int, debug: Optional[MoEDebug] = None,
                      stream=None):
    _check(_lib.nvfp4_moe_forward_w4a16(ctypes.byref(weights), _ptr(x), _ptr(router_logits),
                                        num_tokens, k, _ptr(residual), _ptr(out),
                                        _ptr(workspace), workspace_bytes,
                                        None if debug is None else ctypes.byref(debug),
                                        _stream(stream)), "nvfp4_moe_forward_w4a16")


def quantize_experts_mx(x, ldx: int, K: int, src_row, num_src_rows: int, P: int,
                        expert_offsets, num_experts: int, gscale, codes, sf, stream=None):
    _check(_lib.nvfp4_quantize_experts_mx(_ptr(x), ldx, K, _ptr(src_row), num_src_rows, P,
                                          _ptr(expert_offsets), num_experts, _ptr(gscale),
                                          _ptr(codes), _ptr(sf), _stream(stream)),
           "nvfp4_quantize_experts_mx")


def quantize_pairs_mx(x, ldx: int, num_rows: int, K: int, topk: int, expert_idx, dst_row,
                      num_experts: int, gscale, codes, sf, num_dst_rows: int, stream=None):
    _check(_lib.nvfp4_quantize_pairs_mx(_ptr(x), ldx, num_rows, K, topk, _ptr(expert_idx),
                                        _ptr(dst_row), num_experts, _ptr(gscale), _ptr(codes),
                                        _ptr(sf), num_dst_rows, _stream(stream)),
           "nvfp4_quantize_pairs_mx")


def moe_pack_weights_mx(projection: int, codes, sf, num_experts: int, hidden: int, inter: int,
                        codes_out, sf_out, stream=None):
    _check(_lib.nvfp4_moe_pack_weights_mx(projection, _ptr(codes), _ptr(sf), num_experts, hidden,
                                          inter, _ptr(codes_out), _ptr(sf_out), _stream(stream)),
           "nvfp4_moe_pack_weights_mx")


def moe_forward_mx(weights: MoEWeights, x, router_logits, num_tokens: int, k: int, residual, out,
                   workspace, workspace_bytes: int, debug: Optional[MoEDebug] = None,
                   stream=None):
    _check(_lib.nvfp4_moe_forward_mx(ctypes.byref(weights), _ptr(x), _ptr(router_logits),
                                     num_tokens, k, _ptr(residual), _ptr(out), _ptr(workspace),
                                     workspace_bytes, None if debug is None else ctypes.byref(debug),
                                     _stream(stream)), "nvfp4_moe_forward_mx")


def moe_forward_noalloc(weights: MoEWeights, x, router_logits, num_tokens: int, k: int, residual,
                        out, debug: Optional[MoEDebug] = None, stream=None):
    _check(_lib.nvfp4_moe_forward_noalloc(ctypes.byref(weights), _ptr(x), _ptr(router_logits),
                                          num_tokens, k, _ptr(residual), _ptr(out),
                                          None if debug is None else ctypes.byref(debug),
                                          _stream(stream)), "nvfp4_moe_forward_noalloc")


# The dense operators: pointers are addresses (integers, None for NULL) and the
# stream is a handle, so that a small call pays for no more than the C call.

def rmsnorm(*args):
    """The arguments of nvfp4_rmsnorm, in order."""
    _check_size(args[8], "nvfp4_rmsnorm: num_rows")
    _check_size(args[9], "nvfp4_rmsnorm: K")
    status = _lib.nvfp4_rmsnorm(*args)
    if status != OK:
        raise NVFP4Error(status, "nvfp4_rmsnorm")


def block_norm(p: bytes, stream):
    """p: pack_block_norm's fields of nvfp4_block_norm_t, sizes checked by the caller."""
    status = _lib.nvfp4_block_norm(p, stream)
    if status != OK:
        raise NVFP4Error(status, "nvfp4_block_norm")


def quantize_rows_fp8(*args):
    """The arguments of nvfp4_quantize_rows_fp8, in order."""
    _check_size(args[3], "nvfp4_quantize_rows_fp8: num_rows")
    _check_size(args[4], "nvfp4_quantize_rows_fp8: K")
    status = _lib.nvfp4_quantize_rows_fp8(*args)
    if status != OK:
        raise NVFP4Error(status, "nvfp4_quantize_rows_fp8")


def linear_workspace_size(p: LinearFields) -> int:
    n = ctypes.c_size_t()
    _check(_lib.nvfp4_linear_workspace_size(ctypes.byref(p), ctypes.byref(n)),
           "nvfp4_linear_workspace_size")
    return n.value


def linear(p: LinearFields, workspace, workspace_bytes: int, stream):
    status = _lib.nvfp4_linear(ctypes.byref(p), workspace, workspace_bytes, stream)
    if status != OK:
        raise NVFP4Error(status, "nvfp4_linear")


def linear_w4_workspace_size(p: LinearFields, w4: int) -> int:
    n = ctypes.c_size_t()
    _check(_lib.nvfp4_linear_w4_workspace_size(ctypes.byref(p), w4, ctypes.byref(n)),
           "nvfp4_linear_w4_workspace_size")
    return n.value


def linear_w4(p: LinearFields, w4: int, gain, workspace, workspace_bytes: int, stream):
    status = _lib.nvfp4_linear_w4(ctypes.byref(p), w4, gain, workspace, workspace_bytes, stream)
    if status != OK:
        raise NVFP4Error(status, "nvfp4_linear_w4")


def grouped_linear(p: bytes, stream):
    """p: pack_grouped_linear's fields of nvfp4_grouped_linear_t, sizes checked by the
    caller."""
    status = _lib.nvfp4_grouped_linear(p, stream)
    if status != OK:
        raise NVFP4Error(status, "nvfp4_grouped_linear")


def combine(*args):
    """The arguments of nvfp4_combine, in order."""
    for i, name in ((3, "num_rows"), (6, "num_tokens"), (7, "k"), (8, "H")):
        _check_size(args[i], f"nvfp4_combine: {name}")
    status = _lib.nvfp4_combine(*args)
    if status != OK:
        raise NVFP4Error(status, "nvfp4_combine")
