"""Argument checks of the dense operators, without a GPU: every malformed call
of dense.py raises ValueError, and the C entry points return their error (or
OK for an empty call) before anything is enqueued."""
import ctypes

import numpy as np
import pytest
import torch

from nvfp4_w4a4_expert_amd import _lib as L
from nvfp4_w4a4_expert_amd import dense as D
from oracle import dense as OD

BF16, F16, F32, U8 = torch.bfloat16, torch.float16, torch.float32, torch.uint8
T, K, N = 5, 64, 32


def buf(rows, cols, dtype=BF16):
    return torch.zeros(rows, cols, dtype=dtype)


def on_cpu(call, match="on a GPU"):
    """The well-formed call fails only where it finds no GPU."""
    with pytest.raises(ValueError, match=match):
        call()


def test_well_formed_calls_reach_the_device_check():
    x, w = buf(T, K), torch.zeros(K, dtype=BF16)
    on_cpu(lambda: D.rms_norm(x, w, residual=buf(T, K), weight_offset=1.0, scales="mx"))
    on_cpu(lambda: D.rms_norm(x, residual=x, total_out=x, out=buf(T, K), scales="row"))
    on_cpu(lambda: D.quantize_fp8(x, "row"))
    on_cpu(lambda: D.linear(x, buf(N, K)))
    on_cpu(lambda: D.linear(x, buf(2 * N, K), bias=torch.zeros(2 * N), gated=True, act="silu", residual=buf(T, N, F32),
                            out_dtype="mx"))
    q = D.FP8Rows(buf(T, K, U8), torch.zeros(T))
    on_cpu(lambda: D.linear(q, (buf(N, K, U8), torch.zeros(N))))
    r = buf(T, N)
    on_cpu(lambda: D.linear(x, buf(N, K), residual=r, out=r))
    wide = buf(T, 2 * N)                                     # column ranges of one buffer are apart
    on_cpu(lambda: D.linear(x, buf(N, K), residual=wide[:, :N], out=wide[:, N:]))
    on_cpu(lambda: D.rms_norm(x[:1], residual=x[3:4]))       # one row: its stride does not matter


def norm_args(**kw):
    a = dict(x=buf(T, K), weight=torch.zeros(K, dtype=BF16), residual=buf(T, K), scales="mx")
    a.update(kw)
    x, w = a.pop("x"), a.pop("weight")
    return lambda: D.rms_norm(x, w, **a)


@pytest.mark.parametrize("kw", [
    dict(x=buf(T, K, F32)), dict(x=torch.zeros(T, 2, K, dtype=BF16)), dict(x=None), dict(x=np.zeros((T, K))),
    dict(x=torch.zeros(K, T, dtype=BF16).t()), dict(x=buf(T, K + 4)[:, :K]), dict(x=buf(T, K + 8)[:, 4:4 + K]),
    dict(x=buf(1, K).expand(T, K)), dict(residual=buf(T, K, F16)), dict(residual=buf(T - 1, K)), dict(residual=buf(T, K + 8)),
    dict(weight=torch.zeros(K)), dict(weight=torch.zeros(K + 8, dtype=BF16)), dict(weight=torch.zeros(1, K, dtype=BF16)),
    dict(weight=torch.zeros(2 * K, dtype=BF16)[::2]), dict(scales="fp8"), dict(scales=32), dict(eps=-1e-6), dict(eps=float("nan")),
    dict(eps=float("inf")), dict(weight_offset=float("nan")), dict(want_y=False, out=buf(T, K)),
    dict(residual=None, total_out=buf(T, K)), dict(residual=None, scales=None, want_y=False), dict(out=buf(T, K, F16)),
    dict(out=buf(T + 1, K)), dict(total_out=buf(T, K, F32)),
    dict(x=buf(T, 40), weight=None, residual=None, scales="mx"), dict(x=buf(T, 12), weight=None, residual=None, scales=None),
    dict(x=buf(T, 0), weight=None, residual=None, scales=None), dict(x=buf(1, 32776), weight=None, residual=None, scales=None),
])
def test_norm_refusals(kw):
    with pytest.raises(ValueError, match="^(?!.*on a GPU)"):
        norm_args(**kw)()


def test_overlaps_are_refused():
    big = buf(2 * T, K)
    x = big[:T]
    with pytest.raises(ValueError, match="overlaps"):
        D.rms_norm(x, out=big[1:T + 1])
    with pytest.raises(ValueError, match="overlaps"):
        D.rms_norm(x, residual=buf(T, K), out=x, total_out=x)
    with pytest.raises(ValueError, match="overlaps"):
        D.rms_norm(x, residual=big[T:], total_out=big[T - 1:2 * T - 1])
    o = buf(T, 2 * K)
    with pytest.raises(ValueError, match="overlaps"):
        D.rms_norm(o[:, :K], out=o[:, 8:8 + K])
    with pytest.raises(ValueError, match="overlaps"):
        D.linear(x, buf(K, K), out=x)
    w = buf(T, K)
    with pytest.raises(ValueError, match="overlaps"):
        D.linear(buf(K, K), w, out=torch.as_strided(w, (K, T), (T, 1)))
    r = buf(T + 1, N)
    with pytest.raises(ValueError, match="overlaps"):
        D.linear(x, buf(N, K), residual=r[:T], out=r[1:])


@pytest.mark.parametrize("x,scales", [
    (buf(T, K, F32), "mx"), (buf(T, K), "block"), (buf(T, K), None), (buf(T, 24), "mx"), (buf(T, 4), "row"), (buf(T, 32776), "row"),
    (torch.zeros(K, dtype=BF16), "row")])
def test_quantize_refusals(x, scales):
    with pytest.raises(ValueError, match="^(?!.*on a GPU)"):
        D.quantize_fp8(x, scales)


def q_row(rows, cols=K):
    return D.FP8Rows(buf(rows, cols, U8), torch.zeros(rows))


def q_mx(rows, cols=K):
    return D.FP8Rows(buf(rows, cols, U8), torch.zeros(rows, cols // 32, dtype=U8))


@pytest.mark.parametrize("a,w,kw", [
    (buf(T, K), buf(N, K, F16), {}), (buf(T, K), q_row(N), {}), (q_mx(T), q_row(N), {}), (buf(T, K), buf(N, K + 8), {}),
    (buf(T, K, F32), buf(N, K, F32), {}), (buf(T, 12), buf(N, 12), {}), (buf(T, 0), buf(N, 0), {}), (q_row(T, 24), q_row(N, 24), {}),
    (q_mx(T, 48), q_mx(N, 48), {}), (buf(T, K).t(), buf(N, T), {}), (buf(T, K + 4)[:, :K], buf(N, K), {}),
    ([buf(T, K, U8), torch.zeros(T)], q_row(N), {}), ((buf(T, K, U8),), q_row(N), {}),
    ((buf(T, K, U8), torch.zeros(T + 1)), q_row(N), {}), ((buf(T, K, U8), torch.zeros(T, 1)), q_row(N), {}),
    ((buf(T, K, U8), torch.zeros(T, 2, dtype=torch.int32)), q_mx(N), {}), ((buf(T, K, U8), torch.zeros(2 * T)[::2]), q_row(N), {}),
    ((buf(T, K, torch.int8), torch.zeros(T)), q_row(N), {}),
    (buf(T, K), buf(N, K), dict(act="tanh")), (buf(T, K), buf(N, K), dict(act=["silu"])), (buf(T, K), buf(N, K), dict(gated=1)),
    (buf(T, K), buf(N + 1, K), dict(gated=True)), (buf(T, K), buf(N, K), dict(bias=torch.zeros(N + 1))),
    (buf(T, K), buf(N, K), dict(bias=torch.zeros(N, dtype=torch.float64))), (buf(T, K), buf(N, K), dict(bias=torch.zeros(2 * N)[::2])),
    (buf(T, K), buf(N, K), dict(gated=True, bias=torch.zeros(N // 2))), (buf(T, K), buf(N, K), dict(residual=buf(T, N + 1))),
    (buf(T, K), buf(N, K), dict(residual=buf(N, T).t())), (buf(T, K), buf(N, K), dict(residual=buf(1, N).expand(T, N))),
    (buf(T, K), buf(N, K), dict(residual=buf(T, N, torch.float64))), (buf(T, K), buf(N, K), dict(out_dtype="row")),
    (buf(T, K), buf(N, K), dict(out_dtype=torch.float64)), (buf(T, K), buf(N, K), dict(out_dtype=torch.uint8)),
    (buf(T, K), buf(N - 1, K), dict(out_dtype="mx")), (buf(T, K), buf(N, K), dict(out_dtype="mx", out=buf(T, N, U8))),
    (buf(T, K), buf(N, K), dict(out=buf(T, N), out_dtype=F32)), (buf(T, K), buf(N, K), dict(out=buf(T - 1, N))),
    (buf(T, K), buf(N, K), dict(out=buf(N, T).t())),
])
def test_linear_refusals(a, w, kw):
    with pytest.raises(ValueError, match="^(?!.*on a GPU)"):
        D.linear(a, w, **kw)


# ---- the C entry points -----------------------------------------------------------

GOOD = 4096                                                  # an aligned address no check dereferences


def c_norm(**kw):
    a = dict(type=L.TYPE_BF16, x=GOOD, ldx=64, residual=GOOD, ldr=64, weight=GOOD, offset=1.0, eps=1e-6, rows=0, K=64,
             sum=GOOD, lds=64, y=GOOD, ldy=64, fp8=L.TYPE_FP8_MX, codes=GOOD, scales=GOOD)
    a.update(kw)
    return L._lib.nvfp4_rmsnorm(*a.values(), None)


def test_c_norm_checks():
    assert c_norm() == L.OK                                  # no rows: nothing to do
    assert c_norm(x=None, y=None, codes=None) == L.OK
    for kw in (dict(type=L.TYPE_FP32), dict(type=9), dict(fp8=L.TYPE_BF16), dict(fp8=-2), dict(rows=-1), dict(K=0), dict(K=60),
               dict(K=40), dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf")), dict(offset=float("inf")),
               dict(residual=None)):
        assert c_norm(**kw) == L.ERR_INVALID_ARG, kw
    assert c_norm(K=32800) == L.ERR_UNSUPPORTED
    for kw in (dict(x=None), dict(x=GOOD + 8), dict(ldx=56), dict(ldx=68), dict(residual=GOOD + 2), dict(ldr=72 + 4), dict(weight=GOOD + 8),
               dict(sum=GOOD + 4), dict(lds=63), dict(y=GOOD + 8), dict(ldy=32), dict(codes=None), dict(codes=GOOD + 4),
               dict(scales=None), dict(fp8=L.TYPE_FP8_ROW, scales=GOOD + 2), dict(sum=None, y=None, fp8=L.FP8_NONE)):
        assert c_norm(rows=3, **kw) == L.ERR_INVALID_ARG, kw


def test_c_quantize_checks():
    f = L._lib.nvfp4_quantize_rows_fp8
    assert f(L.TYPE_BF16, None, 64, 0, 64, L.TYPE_FP8_ROW, None, None, None) == L.OK
    good = [L.TYPE_FP16, GOOD, 64, 3, 64, L.TYPE_FP8_MX, GOOD, GOOD]
    for i, v in ((0, L.TYPE_FP32), (1, None), (1, GOOD + 8), (2, 60), (2, 8), (3, -1), (4, 7), (4, 24), (5, L.FP8_NONE), (5, L.TYPE_FP32),
                 (6, None), (6, GOOD + 1), (7, None)):
        bad = list(good)
        bad[i] = v
        assert f(*bad, None) == L.ERR_INVALID_ARG, (i, v)
    good[4], good[2] = 65536, 65536
    assert f(*good, None) == L.ERR_UNSUPPORTED


def c_linear(ws=None, n=0, **kw):
    a = dict(a=GOOD, a_scales=GOOD, w=GOOD, w_scales=GOOD, bias=GOOD, residual=GOOD, out=GOOD, out_scales=GOOD, lda=64, ldw=64,
             ldr=32, ldo=32, M=4, N=32, K=64, type=L.TYPE_FP8_MX, bias_type=L.TYPE_FP32, residual_type=L.TYPE_BF16,
             out_type=L.TYPE_FP8_MX, act=L.ACT_SILU, gated=0)
    a.update(kw)
    return L._lib.nvfp4_linear(ctypes.byref(L.Linear(**a)), ws, n, None)


def test_c_linear_checks():
    assert L._lib.nvfp4_linear(None, None, 0, None) == L.ERR_INVALID_ARG
    assert c_linear(M=0, a=None, out=None) == L.OK and c_linear(N=0, ldo=0) == L.OK
    for kw in (dict(M=-1), dict(N=-1), dict(K=0), dict(K=48), dict(type=L.TYPE_FP8_ROW, K=40), dict(type=L.TYPE_BF16, K=60),
               dict(type=L.TYPE_FP32), dict(type=7), dict(act=-1), dict(act=5), dict(gated=2), dict(out_type=L.TYPE_FP8_ROW),
               dict(out_type=9), dict(bias_type=L.TYPE_FP8_MX), dict(residual_type=L.TYPE_FP8_ROW), dict(N=31, M=4)):
        assert c_linear(**kw) == L.ERR_INVALID_ARG, kw
    for kw in (dict(a=None), dict(w=None), dict(out=None), dict(a=GOOD + 8), dict(w=GOOD + 4), dict(lda=63), dict(lda=72), dict(ldw=32),
               dict(type=L.TYPE_BF16, lda=68), dict(a_scales=None), dict(w_scales=None), dict(type=L.TYPE_FP8_ROW, a_scales=GOOD + 1),
               dict(bias=GOOD + 2), dict(residual=GOOD + 1), dict(ldr=31), dict(ldo=31), dict(out_scales=None), dict(out=GOOD + 8),
               dict(ldo=40), dict(out_type=L.TYPE_FP32, out=GOOD + 2), dict(out_type=L.TYPE_BF16, out=GOOD + 1)):
        assert c_linear(**kw) == L.ERR_INVALID_ARG, kw
    for kw in (dict(K=(1 << 24) + 32, lda=1 << 26, ldw=1 << 26), dict(N=(1 << 24) + 32, ldo=1 << 26, ldr=1 << 26),
               dict(M=1 << 30, N=1 << 20, ldo=1 << 20, ldr=1 << 20), dict(lda=(1 << 23) + 16), dict(ldw=(1 << 23) + 16)):
        assert c_linear(**kw) == L.ERR_UNSUPPORTED, kw


def test_c_linear_workspace_size():
    p, n = L.Linear(M=4, N=32, K=64, type=L.TYPE_BF16), ctypes.c_size_t(7)
    assert L._lib.nvfp4_linear_workspace_size(ctypes.byref(p), ctypes.byref(n)) == L.OK
    assert L._lib.nvfp4_linear_workspace_size(ctypes.byref(p), None) == L.ERR_INVALID_ARG
    assert L._lib.nvfp4_linear_workspace_size(None, ctypes.byref(n)) == L.ERR_INVALID_ARG
    p.K = 20
    assert L._lib.nvfp4_linear_workspace_size(ctypes.byref(p), ctypes.byref(n)) == L.ERR_INVALID_ARG


# ---- the oracle itself --------------------------------------------------------------

def test_oracle_e4m3_agrees_with_torch():
    v = torch.cat([torch.linspace(-448, 448, 20001), torch.logspace(-5, 0, 4000), torch.tensor([0.0, -0.0, 2.0 ** -10, 3 * 2.0 ** -10])])
    want = v.to(torch.float8_e4m3fn).view(U8).numpy()
    assert np.array_equal(OD.e4m3_encode(v.numpy()), want)
    c = np.arange(256, dtype=np.uint8)
    ref = torch.from_numpy(c).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(np.nan_to_num(OD.e4m3_decode(c), nan=9e9), np.nan_to_num(ref, nan=9e9))


def test_oracle_block_scale_is_the_smallest_covering_power():
    for amax in (448.0, 448.0001, 447.9, 1.75, 1.7500001, 3.5, 1e-30, 3e38, 1.0, 2.0 ** -126):
        c = int(OD.block_code(np.array([np.float32(amax)]))[0])
        f = float(np.float32(amax))
        assert f <= 448 * 2.0 ** (c - 127) and (c == 1 or f > 448 * 2.0 ** (c - 128))
    assert OD.block_code(np.array([0.0]))[0] == 1


def test_oracle_quantiser_holds_its_own_bounds():
    x = torch.randn(20, 96, generator=torch.Generator().manual_seed(1)).numpy()
    for q in (OD.quantize_row, OD.quantize_block):
        c, s = q(x)
        OD.check_fp8(c, s, x.astype(np.float64), 0.0)
        bad = c.copy()
        bad[3, 5] += 2 if (bad[3, 5] & 0x7F) < 0x7C else -2
        with pytest.raises(AssertionError):
            OD.check_fp8(bad, s, x.astype(np.float64), 0.0)
