"""Sizes, scales and empty results at the ends of the dense operators' ranges,
without a GPU."""
import ctypes

import numpy as np
import pytest
import torch

from nvfp4_w4a4_expert_amd import _lib as L
from nvfp4_w4a4_expert_amd import dense as D
from oracle import dense as OD

BF16, U8 = torch.bfloat16, torch.uint8
PAST = 2 ** 32                                               # 0 in 32 bits


def meta(rows, cols, dtype=BF16):
    """A tensor of any size without memory."""
    return torch.empty(rows, cols, dtype=dtype, device="meta")


# ---- sizes that 32 bits do not hold ------------------------------------------------

@pytest.mark.parametrize("rows", [2 ** 31, PAST, PAST + 5])
def test_row_counts_past_32_bits_are_refused(rows):
    x = meta(rows, 32)
    w, q = meta(8, 32), (meta(8, 32, U8), torch.empty(8, 1, dtype=U8, device="meta"))
    many = (meta(rows, 32, U8), torch.empty(rows, 1, dtype=U8, device="meta"))
    for call in (lambda: D.rms_norm(x), lambda: D.rms_norm(x, residual=x, scales="mx"), lambda: D.quantize_fp8(x),
                 lambda: D.quantize_fp8(x, "row"), lambda: D.linear(x, w), lambda: D.linear(w, x),
                 lambda: D.linear(w, x, gated=True), lambda: D.linear(many, q), lambda: D.linear(q, many)):
        with pytest.raises(L.NVFP4Error, match=str(rows)) as e:
            call()
        assert e.value.status == L.ERR_UNSUPPORTED


def test_columns_past_32_bits_are_refused():
    with pytest.raises(L.NVFP4Error, match=str(PAST + 64)):
        D.linear(meta(2, PAST + 64), meta(3, PAST + 64))


def test_results_past_the_limit_are_refused_before_they_are_allocated():
    for a, w, kw in ((meta(1 << 30, 64), meta(1 << 20, 64), {}), (meta(1 << 30, 64), meta(1 << 20, 64), dict(gated=True)),
                     (meta(4, 64), meta((1 << 24) + 32, 64), dict(out_dtype="mx")), (meta(2, (1 << 22) + 8), meta(3, (1 << 22) + 8), {})):
        with pytest.raises(L.NVFP4Error) as e:
            D.linear(a, w, **kw)
        assert e.value.status == L.ERR_UNSUPPORTED


def test_last_row_count_of_32_bits_is_taken():
    with pytest.raises(ValueError, match="on a GPU"):
        D.quantize_fp8(meta(2 ** 31 - 1, 32))


@pytest.mark.parametrize("n", [2 ** 31, PAST, PAST + 5, -2 ** 31 - 1])
def test_binding_refuses_sizes_that_it_would_cut(n):
    norm = [L.TYPE_BF16, None, 64, None, 0, None, 0.0, 1e-6, 0, 64, None, 0, None, 64, L.FP8_NONE, None, None, None]
    quant = [L.TYPE_BF16, None, 64, 0, 64, L.TYPE_FP8_MX, None, None, None]
    L.rmsnorm(*norm)                                         # no rows: nothing to do
    L.quantize_rows_fp8(*quant)
    for f, args, places in ((L.rmsnorm, norm, (8, 9)), (L.quantize_rows_fp8, quant, (3, 4))):
        for at in places:
            bad = list(args)
            bad[at] = n
            with pytest.raises(L.NVFP4Error) as e:
                f(*bad)
            assert e.value.status == L.ERR_UNSUPPORTED
    for kw in (dict(M=n), dict(N=n), dict(K=n)):
        with pytest.raises(L.NVFP4Error) as e:
            L.Linear(**kw)
        assert e.value.status == L.ERR_UNSUPPORTED
    with pytest.raises(L.NVFP4Error):
        L.Linear(*[None] * 8, *[64] * 4, n, 32, 64)
    p = L.Linear(M=2 ** 31 - 1, N=0, K=64, type=L.TYPE_BF16)
    assert p.M == 2 ** 31 - 1 and isinstance(p, L.LinearFields) and L.linear_workspace_size(p) == 0
    assert ctypes.sizeof(L.Linear) == ctypes.sizeof(L.LinearFields)


# ---- results without rows ------------------------------------------------------------

def test_dequantize_of_no_rows():
    for scales in (torch.zeros(0, 2, dtype=U8), torch.zeros(0)):
        v = D.FP8Rows(torch.zeros(0, 64, dtype=U8), scales).dequantize()
        assert v.shape == (0, 64) and v.dtype == torch.float32


def test_dequantize_of_strided_codes_and_end_scales():
    codes = torch.arange(3 * 160, dtype=torch.int32).remainder(127).to(U8).view(3, 160)[:, 32:96]
    scales = torch.tensor([[0, 127], [254, 1], [255, 130]], dtype=U8)
    v = D.FP8Rows(codes, scales).dequantize()
    want = codes.contiguous().view(torch.float8_e4m3fn).double().view(3, 2, 32) * (2.0 ** (scales.double() - 127))[..., None]
    want = want.view(3, 64)
    ok = torch.ones(3, 64, dtype=torch.bool)
    ok[2, :32] = False                                       # scale code 255 is NaN
    assert v[~ok].isnan().all() and torch.equal(v[ok], want[ok].float())


# ---- the oracle's cut sums -----------------------------------------------------------

def test_oracle_cut_sums():
    """Exact where no product is more than 5 powers of two below the largest of its
    eight; else the small ones are cut towards zero, by less than 2^-13 of the
    largest each; a cut five bits coarser is far outside the bound."""
    rng = np.random.default_rng(5)
    codes = lambda lo, hi: (rng.integers(lo, hi, (20, 256)) | 128 * rng.integers(0, 2, (20, 256))).astype(np.uint8)
    a, w = OD.e4m3_decode(codes(0x30, 0x40)), OD.e4m3_decode(codes(0x30, 0x40))
    s, err = OD.cut_sums(a, w)
    assert np.array_equal(s, a @ w.T) and err.max() < 1e-3 * np.abs(s).mean()
    a, w = OD.e4m3_decode(codes(0, 0x7F)), OD.e4m3_decode(codes(0, 0x7F))
    s, err = OD.cut_sums(a, w)
    p = np.abs(a[:, None] * w[None]).reshape(20, 20, 32, 8)
    off, coarse = np.abs(s - a @ w.T), np.abs(OD.cut_sums(a, w, bits=8)[0] - s)
    assert np.all(off <= 7 * 2.0 ** -13 * p.max(3).sum(2)) and off.max() > 0
    assert np.median(coarse / err) > 2
    one = np.zeros((1, 8))
    one[0, 0], one[0, 7] = 256.0, 1.125
    assert OD.cut_sums(one, np.abs(one))[0] == 65536 and OD.cut_sums(np.roll(one, 4, 1), -np.abs(np.roll(one, 4, 1)))[0] == -65536


# ---- tensors without strides ---------------------------------------------------------

def test_sparse_tensors_are_refused():
    """As every tensor of a wrong layout: with ValueError."""
    x, w = torch.zeros(4, 64, dtype=BF16), torch.zeros(64, dtype=BF16)
    q = (torch.zeros(4, 64, dtype=U8), torch.zeros(4))
    m = (torch.zeros(4, 64, dtype=U8), torch.zeros(4, 2, dtype=U8))
    sp = lambda t: t.to_sparse()
    for call in (lambda: D.rms_norm(sp(x)), lambda: D.rms_norm(x, sp(w)), lambda: D.rms_norm(x, residual=sp(x)),
                 lambda: D.rms_norm(x, out=sp(x)), lambda: D.quantize_fp8(sp(x)), lambda: D.linear(sp(x), x),
                 lambda: D.linear(x, sp(x)), lambda: D.linear(x, x, bias=sp(torch.zeros(4))),
                 lambda: D.linear(x, x, residual=sp(torch.zeros(4, 4))), lambda: D.linear(x, x, out=sp(torch.zeros(4, 4))),
                 lambda: D.linear((sp(q[0]), q[1]), q), lambda: D.linear(q, (q[0], sp(q[1]))), lambda: D.linear((m[0], sp(m[1])), m)):
        with pytest.raises(ValueError, match="^(?!.*on a GPU)"):
            call()
