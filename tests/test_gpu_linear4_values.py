"""GPU tests of 4-bit weights and values that are not finite: quantize_fp4's refusals,
activations against weights at the end of the range."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

BF16, F16, F32, U8 = torch.bfloat16, torch.float16, torch.float32, torch.uint8


def D():
    from nvfp4_w4a4_expert_amd import dense
    return dense


def rand(shape, seed, dtype=BF16, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale).to(dtype)


@pytest.mark.parametrize("scales", ["nv", "mx"])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), float("-inf")])
def test_quantize_refuses_weights_that_are_not_finite(scales, value):
    for rows, K in ((1, 32), (70, 352)):
        w = rand((rows, K), 1).cuda()
        D().quantize_fp4(w, scales)
        for at in ((0, 0), (rows - 1, K - 1)):
            bad = w.clone()
            bad[at] = value
            with pytest.raises(ValueError, match="finite"):
                D().quantize_fp4(bad, scales)
        # what lies between the rows does not count
        wide = torch.full((rows, K + 16), value, dtype=BF16, device="cuda")
        wide[:, 8:8 + K] = w
        got, ref = D().quantize_fp4(wide[:, 8:8 + K], scales), D().quantize_fp4(w, scales)
        assert torch.equal(got.codes, ref.codes) and torch.equal(got.scales, ref.scales)
    side = torch.cuda.Stream()
    with pytest.raises(ValueError, match="finite"):
        D().quantize_fp4(bad, scales, stream=side)


@pytest.mark.parametrize("scales", ["nv", "mx"])
def test_quantize_of_no_rows_and_of_the_largest_weights(scales):
    q = D().quantize_fp4(torch.zeros(0, 64, dtype=BF16, device="cuda"), scales)
    assert q.codes.shape == (0, 32) and q.scales.shape == (0, 64 // (16 if scales == "nv" else 32))
    assert D().linear(rand((3, 64), 1).cuda(), q).shape == (3, 0)
    # (4 * 2^126, what "mx" makes of bf16's largest numbers, is infinite)
    most = torch.finfo(BF16).max if scales == "nv" else 2.0 ** 126
    w = torch.full((3, 64), most, dtype=BF16, device="cuda")
    assert ((D().quantize_fp4(w, scales).dequantize() - most).abs() <= most * 0.34).all()


@pytest.mark.parametrize("M", [1, 16, 20, 64, 100])
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_infinite_mx_weights_keep_their_formula(M, gated, dtype):
    """One element of every row of w is not 0, in a block of the largest scales: products
    are exact, infinite where they or the element in bf16 pass the range, and a positive a
    meets no NaN; 0 times an infinite element is one."""
    g = np.random.default_rng(M)
    N, K = 84, 416
    at, code, scale = g.integers(0, K, N), g.integers(1, 8, N) + 8 * g.integers(0, 2, N), g.choice([250, 252, 253, 254], N)
    codes = np.zeros((N, K), np.uint8)
    codes[np.arange(N), at] = code
    sf = np.full((N, K // 32), 127, np.uint8)
    sf[np.arange(N), at // 32] = scale
    w = D().FP4Rows(torch.from_numpy(codes[:, 0::2] | codes[:, 1::2] << 4).cuda(), torch.from_numpy(sf).cuda())
    a = torch.from_numpy(g.integers(1, 0x7C00 if dtype == F16 else 0x7F80, (M, K)).astype(np.int16)).view(dtype)
    value = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])[code & 7] * np.where(code & 8, -1.0, 1.0) * 2.0 ** (scale - 127.0)
    value = np.where(np.abs(value) >= 2.0 ** 128, np.copysign(np.inf, value), value)
    with np.errstate(all="ignore"):
        ref = (a.double().numpy()[:, at] * value).astype(np.float32)
    if gated:
        with np.errstate(all="ignore"):
            ref = ref[:, :N // 2] * ref[:, N // 2:]
    got = D().linear(a.cuda(), w, gated=gated, out_dtype=F32).cpu().numpy()
    assert np.array_equal(got, ref, equal_nan=True)
    if not gated:
        a[:, at[0]] = 0.0
        got = D().linear(a.cuda(), w, out_dtype=F32).cpu().numpy()
        with np.errstate(all="ignore"):
            ref = (a.double().numpy()[:, at] * value).astype(np.float32)
        assert np.array_equal(got, ref, equal_nan=True) and np.isnan(ref[:, at == at[0]]).any() == bool(np.isinf(value[at == at[0]]).any())
