"""Argument checks of the experts' operators, without a GPU."""
import numpy as np
import pytest
import torch

from nvfp4_w4a4_expert_amd import _lib as L
from nvfp4_w4a4_expert_amd import experts as X

BF16, F16, F32, I32 = torch.bfloat16, torch.float16, torch.float32, torch.int32
T, TOP, H = 5, 2, 64


def buf(rows, cols, dtype=BF16):
    return torch.zeros(rows, cols, dtype=dtype)


def ints(*shape):
    return torch.zeros(shape, dtype=I32)


def comb(**kw):
    a = dict(values=buf(T * TOP, H), weights=buf(T, TOP, F32), inv_pair=ints(T * TOP))
    a.update(kw)
    v, w, inv = a.pop("values"), a.pop("weights"), a.pop("inv_pair")
    return lambda: X.combine(v, w, inv, **a)


def test_well_formed_calls_reach_the_device_check():
    r = buf(T, H, F32)
    for call in (comb(), comb(values=buf(3, H, F32), inv_pair=ints(T, TOP)), comb(residual=r, out=r), comb(out_dtype=F16, residual=buf(T, H, F16)),
                 lambda: X.route(buf(T, 9, F32), 3), lambda: X.permute(ints(T, 3), 9)):
        with pytest.raises(ValueError, match="on a GPU"):
            call()


@pytest.mark.parametrize("kw", [
    dict(values=None), dict(values=buf(T, H, torch.float64)), dict(values=buf(T, 12)), dict(values=buf(T, 0)), dict(values=buf(T, H + 4)[:, :H]),
    dict(values=buf(H, T).t()), dict(weights=buf(T, TOP)), dict(weights=torch.zeros(T, dtype=F32)), dict(weights=buf(T, 2 * TOP, F32)[:, ::2]),
    dict(weights=buf(T, 0, F32), inv_pair=ints(0)), dict(weights=None), dict(inv_pair=ints(T)), dict(inv_pair=torch.zeros(T * TOP, dtype=torch.int64)),
    dict(inv_pair=ints(2 * T * TOP)[::2]), dict(inv_pair=None), dict(residual=buf(T, H + 8)), dict(residual=buf(T + 1, H)),
    dict(residual=buf(T, H, torch.float64)), dict(out_dtype=torch.int8), dict(out_dtype="mx"), dict(out=buf(T, H, F16), out_dtype=BF16),
    dict(out=buf(T + 1, H)), dict(values=buf(T * TOP, H).to_sparse()), dict(weights=buf(1025 // 1025, 1025, F32), inv_pair=ints(1025)),
])
def test_combine_refusals(kw):
    with pytest.raises(ValueError, match="^(?!.*on a GPU)"):
        comb(**kw)()


def test_combine_overlaps():
    v = buf(2 * T, H)
    with pytest.raises(ValueError, match="overlaps"):
        comb(values=v, out=v[:T])()
    r = buf(T + 1, H)
    with pytest.raises(ValueError, match="overlaps"):
        comb(residual=r[:T], out=r[1:])()


@pytest.mark.parametrize("call", [
    lambda: X.route(buf(T, 9), 2), lambda: X.route(buf(T, 9, F32), 0), lambda: X.route(buf(T, 9, F32), 10), lambda: X.route(buf(T, 40, F32), 33),
    lambda: X.route(buf(T, 1025, F32), 2), lambda: X.route(buf(9, T, F32).t(), 2), lambda: X.route(buf(T, 9, F32), 2.0),
    lambda: X.route(np.zeros((T, 9), np.float32), 2), lambda: X.permute(ints(T), 4), lambda: X.permute(ints(T, 0), 4),
    lambda: X.permute(torch.zeros(T, 2, dtype=torch.int64), 4), lambda: X.permute(ints(T, 2), 0), lambda: X.permute(ints(T, 2), 1025),
    lambda: X.permute(ints(2, T).t(), 4)])
def test_routing_refusals(call):
    with pytest.raises(ValueError, match="^(?!.*on a GPU)"):
        call()


def c_combine(**kw):
    a = dict(type=L.TYPE_BF16, values=256, ldv=H, rows=9, weights=256, inv=256, T=T, k=TOP, H=H, rt=L.TYPE_BF16, r=None, ldr=0, ot=L.TYPE_FP32,
             out=256, ldo=H)
    a.update(kw)
    return L._lib.nvfp4_combine(*a.values(), None)


@pytest.mark.parametrize("kw", [
    dict(type=L.TYPE_FP8_ROW), dict(ot=7), dict(r=256, rt=-1), dict(rows=-1), dict(T=-1), dict(k=0), dict(H=12), dict(H=0), dict(values=None),
    dict(values=8), dict(ldv=H - 8), dict(ldv=H + 4), dict(weights=None), dict(weights=2), dict(inv=None), dict(inv=6), dict(out=None), dict(ldo=H + 2),
    dict(r=8, ldr=H), dict(r=256, ldr=H - 8)])
def test_c_combine_refuses(kw):
    assert c_combine(**kw) == L.ERR_INVALID_ARG


def test_c_combine_limits_and_empty_calls():
    assert c_combine(k=1025) == L.ERR_UNSUPPORTED and c_combine(H=(1 << 24) + 8, ldv=1 << 25) == L.ERR_UNSUPPORTED
    assert c_combine(T=0, values=None, weights=None, inv=None, out=None) == L.OK
