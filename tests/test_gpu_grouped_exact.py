"""GPU tests that 8-bit products grouped by expert are exact before their one rounding,
whatever the result's type and the number of rows."""
import numpy as np
import pytest
import torch

from oracle import dense as OD

pytestmark = pytest.mark.gpu

BF16, F16, F32, U8 = torch.bfloat16, torch.float16, torch.float32, torch.uint8


def D():
    from nvfp4_w4a4_expert_amd import dense
    return dense


def X():
    from nvfp4_w4a4_expert_amd import experts
    return experts


def rows8(shape, seed, scales, scale=1.0):
    """FP8Rows on the GPU and their float64 values."""
    g = torch.Generator().manual_seed(seed)
    v = (torch.randn(shape, generator=g) * scale).to(BF16)
    q = D().quantize_fp8(v.reshape(-1, shape[-1]).cuda(), scales)
    f = OD.dequantize(q.codes.cpu().numpy(), q.scales.cpu().numpy()).reshape(shape)
    return D().FP8Rows(*(t.view(*shape[:-1], *t.shape[1:]) for t in q)), f


def ends(sizes):
    return torch.tensor([0] + list(np.cumsum(sizes)), dtype=torch.int32).cuda()


@pytest.mark.parametrize("scales", ["row", "mx"])
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("sizes,N,K", [([1, 0, 3], 48, 96), ([40, 70, 0, 5], 130, 704), ([300, 0, 200], 1600, 352)])
def test_16_bit_results_are_the_fp32_ones_rounded(scales, gated, sizes, N, K):
    P = sum(sizes)
    a, av = rows8((P, K), 1, scales)
    w, wv = rows8((len(sizes), 2 * N if gated else N, K), 2, scales, K ** -0.5)
    call = lambda out: X().grouped_linear(a, w, ends(sizes), act="silu" if gated else None, gated=gated, out_dtype=out)
    whole = call(F32)
    for dtype in (None, F16):
        assert torch.equal(call(dtype), whole.to(dtype or BF16))
    at = 0
    for e, n in enumerate(sizes):
        if n:
            ref, err = OD.linear(av[at:at + n], wv[e], None, "silu" if gated else None, gated)
            OD.check_rounded(whole[at:at + n].cpu().double().numpy(), ref, err, F32, f"expert {e}")
        at += n


@pytest.mark.parametrize("scales", ["row", "mx"])
@pytest.mark.parametrize("rows", [1, 15, 200])
def test_sums_far_below_their_products(scales, rows):
    """448 * 448 - 448 * 448 + 1 * 1 * 30: every partial sum is a whole number below 2^24,
    so the result is 30 whatever the order."""
    E, N, K = 2, 40, 128
    a, w = torch.zeros(E * rows, K), torch.zeros(E, N, K)
    for b in range(0, K, 32):
        a[:, b], a[:, b + 1], w[:, :, b], w[:, :, b + 1] = 448.0, 448.0, 448.0, -448.0
        a[:, b + 2:b + 32], w[:, :, b + 2:b + 32] = 1.0, 1.0
    e4m3 = lambda t: t.to(torch.float8_e4m3fn).view(U8).cuda()
    one = (lambda *s: torch.ones(s).cuda()) if scales == "row" else (lambda *s: torch.full((*s, K // 32), 127, dtype=U8).cuda())
    for dtype in (BF16, F16, F32):
        got = X().grouped_linear((e4m3(a), one(E * rows)), (e4m3(w), one(E, N)), ends([rows] * E), out_dtype=dtype)
        assert (got == 30.0 * K / 32).all()
