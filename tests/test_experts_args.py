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


# ---- grouped_linear -----------------------------------------------------------------

E, N, K, P = 3, 32, 64, 10
U8 = torch.uint8


def w16(*shape, dtype=BF16):
    return torch.zeros(shape or (E, N, K), dtype=dtype)


def grp(**kw):
    a = dict(a=buf(P, K), w=w16(), offsets=ints(E + 1))
    a.update(kw)
    x, w, o = a.pop("a"), a.pop("w"), a.pop("offsets")
    return lambda: X.grouped_linear(x, w, o, **a)


def f8(rows, row=True):
    return buf(rows, K, U8), torch.zeros(rows) if row else buf(rows, K // 32, U8)


def f8w(row=True):
    return torch.zeros(E, N, K, dtype=U8), torch.zeros(E, N) if row else torch.zeros(E, N, K // 32, dtype=U8)


@pytest.mark.parametrize("kw", [
    {}, dict(a=buf(P, K, F16), w=w16(dtype=F16), out_dtype="mx"), dict(a=f8(P), w=f8w()), dict(a=f8(P, False), w=f8w(False), gated=True),
    dict(index=ints(7), index_div=2), dict(index=ints(0)), dict(bias=torch.zeros(E, N), act="gelu"), dict(w=w16(E, N, K + 8)[:, :, :K]),
    dict(w=w16(2 * E, N, K)[::2]), dict(w=w16(1, N, K).expand(1, N, K), offsets=ints(2)), dict(out=buf(P, N, F32)),
    dict(index=ints(7), out=buf(7, N)), dict(w=w16(1024, 2, K), offsets=ints(1025))])
def test_well_formed_grouped_calls(kw):
    with pytest.raises(ValueError, match="on a GPU"):
        grp(**kw)()


@pytest.mark.parametrize("kw", [
    dict(a=None), dict(a=buf(P, K, F32)), dict(a=buf(P, K, F16)), dict(w=buf(N, K)), dict(w=w16(E, N, K + 8)), dict(w=w16(0, N, K), offsets=ints(1)),
    dict(w=w16(1025, 2, K), offsets=ints(1026)), dict(w=w16(E, K, N).transpose(1, 2)), dict(w=w16(1, N, K).expand(E, N, K)),
    dict(w=w16(E, 1, K).expand(E, N, K)), dict(w=w16(E, N, K + 4)[:, :, :K]), dict(w=f8w()), dict(a=f8(P)), dict(a=f8(P), w=f8w(False)),
    dict(a=f8(P, False), w=f8w()), dict(a=f8(P), w=(f8w()[0], torch.zeros(E, N + 1))), dict(a=f8(P), w=(f8w()[0], torch.zeros(2, E, N)[0].t().contiguous().t())),
    dict(w=w16().to_sparse()), dict(offsets=ints(E)), dict(offsets=torch.zeros(E + 1, dtype=torch.int64)), dict(offsets=ints(2 * E + 2)[::2]),
    dict(offsets=None), dict(index=ints(2, 5)), dict(index=torch.zeros(7, dtype=torch.int64)), dict(index=[1, 2]), dict(index=ints(14)[::2]),
    dict(index_div=0), dict(index_div=2.0), dict(index_div=2 ** 31), dict(bias=torch.zeros(N)), dict(bias=torch.zeros(E, N, dtype=torch.float64)),
    dict(bias=torch.zeros(E, 2 * N)[:, ::2]), dict(act="tanh"), dict(gated=1), dict(w=w16(E, N + 1, K), gated=True), dict(out_dtype="row"),
    dict(out_dtype=torch.int8), dict(out_dtype="mx", out=buf(P, N)), dict(w=w16(E, 8, K), out_dtype="mx"), dict(out=buf(P + 1, N)),
    dict(out=buf(P, N), index=ints(7)), dict(out=buf(P, N, F16), out_dtype=BF16), dict(a=buf(P, 12), w=w16(E, N, 12))])
def test_grouped_refusals(kw):
    with pytest.raises(ValueError, match="^(?!.*on a GPU)"):
        grp(**kw)()


def test_grouped_overlaps():
    x = buf(P, K)
    with pytest.raises(ValueError, match="overlaps"):
        grp(a=x, w=w16(E, K, K), out=x)()
    w = w16()
    with pytest.raises(ValueError, match="overlaps"):
        grp(w=w, out=w.view(-1)[:P * N].view(P, N))()


def c_grouped(**kw):
    import ctypes
    f = dict(a=256, w=256, offsets=256, out=256, lda=K, ldw=K, w_each=N * K, ldo=N, num_rows=P, a_rows=P, num_experts=E, N=N, K=K, index_div=1,
             type=L.TYPE_BF16, bias_type=0, out_type=L.TYPE_BF16, act=0, gated=0)
    f.update(kw)
    p = L.GroupedLinear(**f)
    return L._lib.nvfp4_grouped_linear(ctypes.byref(p), None)


@pytest.mark.parametrize("kw", [
    dict(num_rows=-1), dict(a_rows=-1), dict(num_experts=0), dict(type=L.TYPE_FP32), dict(out_type=L.TYPE_FP8_ROW), dict(act=9), dict(gated=2),
    dict(K=12), dict(K=0), dict(N=-1), dict(out_type=L.TYPE_FP8_MX, N=40), dict(a_rows=P - 1), dict(index=256, index_div=0), dict(bias=256, bias_type=4),
    dict(a=None), dict(w=None), dict(out=None), dict(offsets=None), dict(a=264), dict(w=264), dict(offsets=258), dict(index=258), dict(lda=K - 8),
    dict(ldw=K + 4), dict(w_each=N * K - 8), dict(w_each=N * K + 4), dict(type=L.TYPE_FP8_ROW), dict(type=L.TYPE_FP8_ROW, a_scales=258, w_scales=256),
    dict(bias=258, bias_type=L.TYPE_FP32), dict(ldo=N - 1), dict(out=257), dict(out_type=L.TYPE_FP8_MX), dict(out_type=L.TYPE_FP8_MX, out_scales=256, ldo=N + 1)])
def test_c_grouped_refuses(kw):
    assert c_grouped(**kw) == L.ERR_INVALID_ARG


def test_c_grouped_limits_and_empty_calls():
    null = dict(a=None, w=None, offsets=None, out=None)
    for kw in (dict(num_experts=1025), dict(K=(1 << 22) + 8), dict(N=(1 << 24) + 1), dict(num_rows=(1 << 29) + 1, a_rows=(1 << 29) + 1),
               dict(num_rows=1 << 29, a_rows=1 << 29, N=1 << 20), dict(lda=(1 << 22) + 8), dict(ldw=(1 << 22) + 8, w_each=1 << 40)):
        assert c_grouped(**kw) == L.ERR_UNSUPPORTED, kw
    for kw in (dict(num_rows=0), dict(N=0), dict(a_rows=0, index=None, num_rows=0), dict(a_rows=0, index=256)):
        assert c_grouped(**{**null, **kw}) == L.OK, kw
