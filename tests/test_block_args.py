"""Argument checks of block_norm, without a GPU."""
import ctypes

import numpy as np
import pytest
import torch

from nvfp4_w4a4_expert_amd import _lib as L
from nvfp4_w4a4_expert_amd import dense as D

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
T, K = 5, 64


def buf(rows, cols, dtype=BF16):
    return torch.zeros(rows, cols, dtype=dtype)


def args(**kw):
    a = dict(x=buf(T, K), residual=buf(T, K), weight=torch.zeros(K, dtype=BF16), post_weight=torch.zeros(K, dtype=BF16), scales="mx")
    a.update(kw)
    x, r = a.pop("x"), a.pop("residual")
    return lambda: D.block_norm(x, r, **a)


GOOD = [
    {}, dict(gate=0.5), dict(gate=2), dict(gate=torch.zeros(T, 1)), dict(gate=torch.zeros(K, dtype=BF16), gate_act="tanh"),
    dict(gate=torch.zeros(1, K)), dict(gate=buf(T, K), gate_act="sigmoid"), dict(gate=torch.zeros(1)), dict(gate=buf(T, K + 8)[:, :K]),
    dict(gate=buf(T, 7)[:, 3:4]), dict(gate=buf(1, K).expand(T, K)), dict(post_norm=False, post_weight=None), dict(weight=None, scales=None, want_y=False),
    dict(scales="row", want_y=False), dict(residual_scale=-2, weight_offset=1.0), dict(x=buf(1, K), residual=buf(9, K)[3:4], gate=torch.zeros(1, 1)),
]


@pytest.mark.parametrize("kw", GOOD)
def test_well_formed_calls_reach_the_device_check(kw):
    with pytest.raises(ValueError, match="on a GPU"):
        args(**kw)()


def test_outputs_over_inputs():
    x, r = buf(T, K), buf(T, K)
    for kw in (dict(out=x, total_out=r), dict(out=r, total_out=x), dict(total_out=x)):
        with pytest.raises(ValueError, match="on a GPU"):
            D.block_norm(x, r, **kw)
    g = buf(T, K)
    for kw in (dict(out=x, total_out=x), dict(out=g, gate=g), dict(total_out=g, gate=g)):
        with pytest.raises(ValueError, match="overlaps"):
            D.block_norm(x, r, **kw)
    big = buf(2 * T, K)
    with pytest.raises(ValueError, match="overlaps"):
        D.block_norm(big[:T], r, total_out=big[1:T + 1])


@pytest.mark.parametrize("kw", [
    dict(x=buf(T, K, F32)), dict(x=None), dict(x=np.zeros((T, K))), dict(x=buf(K, T).t()), dict(x=buf(T, K + 4)[:, :K]),
    dict(residual=None), dict(residual=buf(T, K, F16)), dict(residual=buf(T - 1, K)), dict(residual=buf(T, K + 8)),
    dict(weight=torch.zeros(K)), dict(weight=torch.zeros(K + 8, dtype=BF16)), dict(post_weight=torch.zeros(1, K, dtype=BF16)),
    dict(post_norm=1), dict(post_norm=False), dict(scales=None, want_y=False), dict(scales="fp8"), dict(eps=-1.0), dict(eps=float("nan")),
    dict(weight_offset=float("inf")), dict(residual_scale=float("nan")), dict(gate=float("inf")), dict(gate="all"), dict(gate=[1.0]),
    dict(gate_act="sigmoid"), dict(gate=0.5, gate_act="tanh"), dict(gate=buf(T, K), gate_act="relu"), dict(gate=buf(T, K), gate_act=["tanh"]),
    dict(gate=buf(T, K, F16)), dict(gate=torch.zeros(T, K, dtype=torch.float64)), dict(gate=torch.zeros(T)), dict(gate=torch.zeros(2, K)),
    dict(gate=torch.zeros(T, 2)), dict(gate=torch.zeros(T, 1, 1)), dict(gate=torch.zeros(())), dict(gate=torch.zeros(2 * K)[::2]),
    dict(gate=buf(T, K + 4)[:, :K]), dict(gate=torch.zeros(K + 1)[1:]), dict(gate=buf(T, 1).to_sparse()), dict(gate=buf(T, K).to_sparse()),
    dict(x=buf(T, K).to_sparse()), dict(residual=buf(T, K).to_sparse()), dict(out=buf(T, K), want_y=False), dict(out=buf(T, K, F16)),
    dict(total_out=buf(T + 1, K)), dict(stream="other"),
])
def test_refusals(kw):
    with pytest.raises(ValueError):
        args(**kw)()
    if "stream" not in kw:
        with pytest.raises(ValueError, match="^(?!.*on a GPU)"):
            args(**kw)()


def fields(**kw):
    p = L.BlockNorm(x=256, residual=512, total_out=1024, y_out=2048, ldx=K, ldr=K, ldt=K, ldy=K, num_rows=T, K=K, type=L.TYPE_BF16, post=1,
                    fp8=L.FP8_NONE, eps=1e-6, gate_scale=1.0, residual_scale=1.0)
    for name, v in kw.items():
        setattr(p, name, v)
    return p


@pytest.mark.parametrize("kw", [
    dict(type=L.TYPE_FP32), dict(num_rows=-1), dict(K=12), dict(K=0), dict(post=2), dict(fp8=L.TYPE_BF16), dict(x=None), dict(residual=None),
    dict(x=264), dict(ldx=K - 8), dict(ldr=K + 4), dict(eps=-1.0), dict(eps=float("inf")), dict(gate_scale=float("nan")),
    dict(residual_scale=float("inf")), dict(weight_offset=float("nan")), dict(total_out=None, y_out=None), dict(weight=8), dict(post_weight=8),
    dict(gate=256, gate_cols=2), dict(gate=256, gate_cols=K, gate_act=3), dict(gate=256, gate_cols=K, gate_type=L.TYPE_FP16),
    dict(gate=256, gate_cols=K, ldg=-8), dict(gate=256, gate_cols=K, ldg=K - 8), dict(gate=256, gate_cols=K, ldg=K + 4),
    dict(gate=258, gate_cols=K), dict(gate=257, gate_cols=1), dict(fp8=L.TYPE_FP8_MX), dict(fp8=L.TYPE_FP8_ROW, codes=256, scales=257),
    dict(total_out=1032), dict(ldt=K - 1), dict(ldy=K + 1),
])
def test_c_entry_refuses(kw):
    assert L._lib.nvfp4_block_norm(ctypes.byref(fields(**kw)), None) == L.ERR_INVALID_ARG


def test_c_entry_limits_and_empty_calls():
    assert L._lib.nvfp4_block_norm(None, None) == L.ERR_INVALID_ARG
    assert L._lib.nvfp4_block_norm(ctypes.byref(fields(K=32776, ldx=32776, ldr=32776, ldt=32776, ldy=32776)), None) == L.ERR_UNSUPPORTED
    assert L._lib.nvfp4_block_norm(ctypes.byref(fields(num_rows=0, x=None, residual=None)), None) == L.OK


def test_packed_fields_are_the_structures():
    """The byte forms of the calls hold every field where the structure has it."""
    for cls, pack in ((L.BlockNorm, L.pack_block_norm), (L.GroupedLinear, L.pack_grouped_linear)):
        values = [(i + 1) * 3 if t is not ctypes.c_float else i + 0.5 for i, (_, t) in enumerate(cls._fields_)]
        data = pack(*values)
        assert len(data) == ctypes.sizeof(cls)
        got = cls.from_buffer_copy(data)
        assert [getattr(got, name) for name, _ in cls._fields_] == values
