"""Argument checks of linear with 4-bit weights and of quantize_fp4, without a GPU."""
import ctypes

import pytest
import torch

from nvfp4_w4a4_expert_amd import _lib as L
from nvfp4_w4a4_expert_amd import dense as D

BF16, F16, F32, U8 = torch.bfloat16, torch.float16, torch.float32, torch.uint8
M, N, K = 5, 32, 64


def buf(rows, cols, dtype=BF16):
    return torch.zeros(rows, cols, dtype=dtype)


def w4(rows=N, cols=K, per=16, scale=None, codes=None, scales=None):
    return D.FP4Rows(buf(rows, cols // 2, U8) if codes is None else codes, buf(rows, cols // per, U8) if scales is None else scales, scale)


@pytest.mark.parametrize("a,w,kw", [
    (buf(M, K), w4(), {}), (buf(M, K, F16), w4(per=32), {}), (buf(M, K), w4(scale=torch.ones(1)), dict(out_dtype="mx")),
    (buf(M, K), w4(scale=torch.ones(())), dict(gated=True, act="silu", bias=torch.zeros(N))), (buf(200, K), w4(), dict(residual=buf(200, N))),
    (buf(M, K), w4(codes=buf(N, 64, U8)[:, :32]), dict(out=buf(M, N, F32)))])
def test_well_formed_calls_reach_the_device_check(a, w, kw):
    with pytest.raises(ValueError, match="on a GPU"):
        D.linear(a, w, **kw)


@pytest.mark.parametrize("a,w,kw", [
    (buf(M, K, F32), w4(), {}), (D.FP8Rows(buf(M, K, U8), torch.zeros(M)), w4(), {}), (buf(M, K + 32), w4(), {}), (buf(M, 48), w4(cols=48), {}),
    (buf(M, K), w4(scales=buf(N, 3, U8)), {}), (buf(M, K), w4(scales=buf(N + 1, K // 16, U8)), {}), (buf(M, K), w4(scales=buf(N, K // 16, F32)), {}),
    (buf(M, K), w4(scales=buf(N, 2 * K // 16, U8)[:, ::2]), {}), (buf(M, K), w4(codes=buf(N, K // 2, torch.int8)), {}),
    (buf(M, K), w4(codes=buf(K // 2, N, U8).t()), {}), (buf(M, K), w4(codes=buf(N, 40, U8)[:, :32]), {}), (buf(M, K), w4(scale=1.0), {}),
    (buf(M, K), w4(scale=torch.ones(2)), {}), (buf(M, K), w4(scale=torch.ones(1, dtype=F16)), {}), (buf(M, K), w4(rows=N + 1), dict(gated=True)),
    (buf(M, K), w4(scales=torch.zeros(N * 4 + 1, dtype=U8)[1:].view(N, 4)), {}), (buf(M, K), w4(codes=buf(N, K // 2, U8).to_sparse()), {}),
    (buf(M, K), w4(scales=buf(N, 4, U8).to_sparse()), {}), (buf(M, K), w4(), dict(act="tanh")), (buf(M, K), w4(), dict(bias=torch.zeros(N + 1))),
    (buf(M, K), w4(rows=40), dict(out_dtype="mx")), (buf(M, K), D.FP4Rows(None, None), {}), (w4(), w4(), {}), (w4(), buf(N, K), {}),
    (buf(M, K), tuple(w4()), {})])
def test_refusals(a, w, kw):
    with pytest.raises(ValueError, match="^(?!.*on a GPU)"):
        D.linear(a, w, **kw)


def test_overlaps():
    codes = buf(N, K // 2, U8)
    with pytest.raises(ValueError, match="overlaps"):
        D.linear(buf(M, K), w4(codes=codes), out=codes.view(-1)[:M * N * 2].view(BF16).view(M, N)[:, :N])
    s = torch.zeros(M * N)
    with pytest.raises(ValueError, match="overlaps"):
        D.linear(buf(M, K), w4(scale=s[3:4]), out=s.view(M, N))


@pytest.mark.parametrize("w,kw", [(buf(N, K, F16), {}), (buf(N, K, F32), {}), (buf(N, 48), {}), (buf(N, 0), {}), (torch.zeros(K, dtype=BF16), {}),
                                  (buf(N, K), dict(scales="row")), (buf(N, K), dict(scales=None)), (buf(K, N).t(), {})])
def test_quantize_refusals(w, kw):
    with pytest.raises(ValueError, match="^(?!.*on a GPU)"):
        D.quantize_fp4(w, **kw)


def fields(**kw):
    f = dict(a=256, w=256, w_scales=256, out=256, lda=K, ldw=K // 2, ldo=N, M=M, N=N, K=K, type=L.TYPE_BF16, out_type=L.TYPE_BF16)
    f.update(kw)
    return L.LinearFields(**f)


def call(w4=L.W4_NV, gain=None, ws=None, n=0, **kw):
    return L._lib.nvfp4_linear_w4(ctypes.byref(fields(**kw)), w4, gain, ws, n, None)


@pytest.mark.parametrize("kw", [
    dict(w4=2), dict(w4=-1), dict(type=L.TYPE_FP8_ROW), dict(type=L.TYPE_FP32), dict(K=48), dict(K=0), dict(M=-1), dict(act=7), dict(gated=3),
    dict(out_type=L.TYPE_FP8_ROW), dict(a=None), dict(w=None), dict(w_scales=None), dict(out=None), dict(a=264), dict(w=264), dict(w_scales=257),
    dict(gain=258), dict(lda=K - 8), dict(lda=K + 4), dict(ldw=K // 2 - 16), dict(ldw=K // 2 + 8), dict(ldo=N - 1), dict(bias=256, bias_type=9),
    dict(residual=256, ldr=N - 1), dict(out_type=L.TYPE_FP8_MX)])
def test_c_entry_refuses(kw):
    assert call(**kw) == L.ERR_INVALID_ARG


def test_c_entry_limits_workspace_and_empty_calls():
    for kw in (dict(K=(1 << 22) + 32), dict(N=(1 << 24) + 1), dict(K=(1 << 21) + 32, type=L.TYPE_FP16, w4=L.W4_MX), dict(lda=(1 << 22) + 8),
               dict(ldw=(1 << 23) + 16), dict(N=1 << 24, K=1 << 13), dict(M=1 << 26, K=512, N=32)):
        assert call(**kw) == L.ERR_UNSUPPORTED, kw
    assert L._lib.nvfp4_linear_w4(None, 0, None, None, 0, None) == L.ERR_INVALID_ARG
    n = ctypes.c_size_t(7)
    assert L._lib.nvfp4_linear_w4_workspace_size(ctypes.byref(fields()), 0, ctypes.byref(n)) == L.OK and n.value == 0
    assert L._lib.nvfp4_linear_w4_workspace_size(ctypes.byref(fields()), 0, None) == L.ERR_INVALID_ARG
    big = fields(M=5000, N=3000, K=640)
    assert L._lib.nvfp4_linear_w4_workspace_size(ctypes.byref(big), 0, ctypes.byref(n)) == L.OK and n.value >= 3000 * 640 * 2
    for ws, size in ((None, n.value), (256, n.value - 1), (264, n.value)):
        assert call(ws=ws, n=size, M=5000, N=3000, K=640, lda=640, ldw=320, ldo=3000) == L.ERR_WORKSPACE
    for kw in (dict(M=0), dict(N=0)):
        assert call(a=None, w=None, out=None, w_scales=None, **kw) == L.OK
