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
