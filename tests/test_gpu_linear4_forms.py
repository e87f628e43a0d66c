"""GPU tests of every kernel of the linear operator with 4-bit weights, at the sizes of
linear4_cases.py, on operands whose sums are exact in fp32: a holds integers up to 3, w
multiples of 1/4 up to 12, K is at most 8224, so a sum is a multiple of 1/4 below 2^19 (21
bits) in any order.  Results equal the float64 ones to the bit, rounded once."""
import pytest
import torch

import linear4_cases as C
from oracle import dense as OD

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
F32, F64, U8 = torch.float32, torch.float64, torch.uint8


def D():
    from nvfp4_w4a4_expert_amd import dense
    return dense


def operands(rows, M, K, scales, dtype, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    draw = lambda lo, hi, *shape: torch.randint(lo, hi, shape, generator=g, device="cuda")
    a = draw(-3, 4, M, K).to(dtype)
    codes = draw(0, 256, rows, K // 2).to(U8)
    if scales == "nv":
        sf = (0x30 + 8 * draw(0, 3, rows, K // 16)).to(U8)     # 1/2, 1, 2
    else:
        sf = draw(126, 129, rows, K // 32).to(U8)
    w = D().FP4Rows(codes, sf, torch.full((1,), 0.5, device="cuda"))
    return a, w, draw(-40, 41, rows).to(F32), lambda *s: draw(-100, 101, *s).to(F32)


def sums(a, w, bias):
    """act's arguments in fp32 (exact)."""
    v = a.to(F64) @ w.dequantize().to(F64).t().contiguous() + bias.to(F64)
    assert torch.equal(v.to(F32).to(F64), v)
    return v.to(F32)


CASES = list(C.all_cases())


@pytest.mark.parametrize("case", CASES, ids=["-".join(map(str, c)) for c in CASES])
def test_every_kernel(case):
    scales, dtype, form, fm, how, M, N, K, gated = case
    rows = 2 * N if gated else N
    a, w, bias, more = operands(rows, M, K, scales, TYPES[dtype], M + N)
    v = sums(a, w, bias)
    if gated:
        ref, r = v[:, :N] * v[:, N:], None
    else:
        r = more(M, N)
        ref = v + r                                            # (exact as well)
    call = lambda out: D().linear(a, w, bias=bias, gated=gated, residual=r, out_dtype=out)
    got = call(F32)
    assert torch.equal(got, ref)
    assert torch.equal(call(F32), got)
    assert torch.equal(call(None), ref.to(TYPES[dtype]))
    if how != "both" and N >= 32 and M * N < 4e6:
        # 8-bit results of whole blocks of columns
        n = N // 32 * 32
        pick = lambda t: torch.cat([t[:n], t[N:N + n]]).contiguous() if gated else t[:n].contiguous()
        q = D().FP4Rows(pick(w.codes), pick(w.scales), w.scale)
        got = D().linear(a, q, bias=pick(bias), gated=gated, out_dtype="mx")
        x = (ref if gated else v)[:, :n].contiguous()
        codes, s = OD.quantize_block(x.cpu().numpy())
        assert torch.equal(got.codes.cpu(), torch.from_numpy(codes)) and torch.equal(got.scales.cpu(), torch.from_numpy(s))
