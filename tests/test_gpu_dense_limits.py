"""GPU tests of the dense operators at the ends of their ranges: scales near the
ends of fp32's and UE8M0's, sums that cancel, results that are small beside
their arguments, launches of more rows than one grid holds, calls from several
threads.  Against the float64 oracle, with bounds derived there or here."""
import numpy as np
import pytest
import torch

from oracle import dense as OD

pytestmark = pytest.mark.gpu

BF16, F16, F32, U8 = torch.bfloat16, torch.float16, torch.float32, torch.uint8


def D():
    from nvfp4_w4a4_expert_amd import dense
    return dense


def f64(t):
    return t.detach().cpu().double().numpy()


# ---- row scales near the ends of fp32's range ----------------------------------------

def row_codes(rows, K, rng, zero=(), low=0x20, high=0x50):
    """Random E4M3 codes of either sign (by default +-(2^-3 to 7.5)), rows `zero` all 0."""
    c = (rng.integers(low, high, (rows, K)) | 128 * rng.integers(0, 2, (rows, K))).astype(np.uint8)
    c[list(zero)] = 0
    return c


def rows_fp8(codes, scales):
    s = np.resize(np.asarray(scales, np.float32), codes.shape[0])
    return D().FP8Rows(torch.from_numpy(codes).cuda(), torch.from_numpy(s).cuda()), OD.dequantize(codes, s)


# scales of a, of w, codes.  The first set's products of two scales are subnormal (a
# few bits) under sums around 1e6, the others' scales lie at both ends of the range
SCALES = [([1e-21, 3e-23, 2.0 ** -70, 2e-21], [1e-22, 4e-22, 1e-23], (0x60, 0x7F)),
          ([1e-30, 2e-38, 1e-44, 7e-42], [3e30, 1e37, 1.5e25], (0x20, 0x50)),
          ([1e30, 3e37, 1e22], [1e-44, 3e-38, 1e-25, 2.0 ** -149], (0x20, 0x50))]


@pytest.mark.parametrize("M,N,K", [(5, 33, 64), (16, 70, 4224), (40, 96, 64), (130, 160, 96), (300, 320, 64), (33, 77, 2832)])
@pytest.mark.parametrize("which", range(len(SCALES)))
def test_row_scale_range(M, N, K, which):
    rng = np.random.default_rng(M + which)
    sa, sw, codes = SCALES[which]
    a, av = rows_fp8(row_codes(M, K, rng, (2,), *codes), sa)
    w, wv = rows_fp8(row_codes(2 * N, K, rng, (1, N + 5), *codes), sw)
    for out in (F32, BF16):
        ref, err = OD.linear(av, wv, scaled=out != F32)
        got = D().linear(a, w, out_dtype=out)
        OD.check_rounded(f64(got), ref, err + 2.0 ** -149, out, f"{M}x{N}x{K}")
    # gated: tiny or huge scales on both factors, the bias brings them to about 1
    b = torch.from_numpy(rng.standard_normal(2 * N).astype(np.float32))
    ref, err = OD.linear(av, wv, f64(b), "relu", True)
    got = D().linear(a, w, bias=b.cuda(), act="relu", gated=True, out_dtype=F32)
    ok = np.abs(ref) < 1e38
    OD.check_rounded(f64(got)[ok], ref[ok], err[ok] + 2.0 ** -148, F32, "gated")


@pytest.mark.parametrize("M", [5, 40, 130, 300])
def test_small_and_zero_sums_under_huge_row_scales(M):
    """Sums of 0 stay 0 and a sum of 2^-10 keeps its value where the product of the
    scales is infinite."""
    N, K = 70, 64
    ca, cw = np.zeros((M, K), np.uint8), np.zeros((N, K), np.uint8)
    ca[:, 3], cw[::2, 3] = 0x10, 0x10                          # 2^-5 each; odd columns are 0
    a, av = rows_fp8(ca, [1e21, 3e24, 1e18])
    w, wv = rows_fp8(cw, [1e18, 1e20, 1.7e16])
    ref, err = OD.linear(av, wv)
    for out in (F32, BF16):
        got = f64(D().linear(a, w, out_dtype=out))
        ok = np.abs(ref) < 3.3e38
        assert ok[:, 1::2].all() and not ref[:, 1::2].any()
        OD.check_rounded(got[ok], ref[ok], err[ok], out)
        assert np.all(np.isinf(got[~ok]))
    b = torch.ones(N)
    got = D().linear(a, w, bias=b.cuda(), out_dtype=F32)
    assert (got[:, 1::2] == 1).all()


# ---- results without rows --------------------------------------------------------------

def test_empty_results_dequantize():
    x = torch.zeros(0, 64, dtype=BF16, device="cuda")
    w = torch.zeros(32, 64, dtype=BF16, device="cuda")
    for r, cols in ((D().rms_norm(x, scales="mx").fp8, 64), (D().rms_norm(x, scales="row").fp8, 64), (D().quantize_fp8(x, "mx"), 64),
                    (D().quantize_fp8(x, "row"), 64), (D().linear(x, w, out_dtype="mx"), 32)):
        assert r.dequantize().shape == (0, cols)
