"""GPU tests of every tile of the products grouped by expert at the sizes of
grouped_cases.py, on operands whose sums are exact in fp32: integers up to 3 and 4 and row
or block scales of 1/2, 1 and 2, K at most 2848, so a sum is a multiple of 1/4 below 2^18
(20 bits) in any order.  Results equal the float64 ones to the bit, rounded once."""
import pytest
import torch

import grouped_cases as C
from oracle import dense as OD

pytestmark = pytest.mark.gpu

BF16, F16, F32, F64, U8, I32 = torch.bfloat16, torch.float16, torch.float32, torch.float64, torch.uint8, torch.int32


def D():
    from nvfp4_w4a4_expert_amd import dense
    return dense


def X():
    from nvfp4_w4a4_expert_amd import experts
    return experts


def operand(draw, most, kind, *shape):
    """(operand, its values in float64)"""
    v = draw(-most, most + 1, *shape)
    if kind in ("bf16", "fp16"):
        return v.to(BF16 if kind == "bf16" else F16), v.to(F64)
    codes = v.to(F32).to(torch.float8_e4m3fn).view(U8)
    if kind == "row":
        s = 2.0 ** draw(-1, 2, *shape[:-1]).to(F32)
        return D().FP8Rows(codes, s), v.to(F64) * s[..., None].to(F64)
    s = draw(126, 129, *shape[:-1], shape[-1] // 32)
    return D().FP8Rows(codes, s.to(U8)), v.to(F64) * (2.0 ** (s - 127).to(F64)).repeat_interleave(32, -1)


CASES = list(C.all_cases())


@pytest.mark.parametrize("case", CASES, ids=["-".join(map(str, c)) for c in CASES])
def test_every_tile(case):
    kind, tile, K, gated, gathered = case
    sizes, N, Ng = C.TILES[tile]
    N, P, E = Ng if gated else N, sum(sizes), len(sizes)
    rows, T = 2 * N if gated else N, P // 2 + 1 if gathered else P
    g = torch.Generator(device="cuda").manual_seed(K)
    draw = lambda lo, hi, *shape: torch.randint(lo, hi, shape, generator=g, device="cuda")
    a, av = operand(draw, 3, kind, T, K)
    w, wv = operand(draw, 4, kind, E, rows, K)
    bias = draw(-9, 10, E, rows).to(F32)
    index = draw(0, 2 * T, P).to(I32) if gathered else None
    offsets = torch.tensor([0] + sizes).cumsum(0).to(I32).cuda()
    at = av[index // 2] if gathered else av
    parts = [x @ wv[e].t().contiguous() + bias[e].to(F64) for e, x in enumerate(at.split(sizes))]
    v = torch.cat(parts)
    assert torch.equal(v.to(F32).to(F64), v)
    ref = v.to(F32)
    if gated:
        ref = ref[:, :N] * ref[:, N:]
    call = lambda out: X().grouped_linear(a, w, offsets, index=index, index_div=2, bias=bias, gated=gated, out_dtype=out)
    got = call(F32)
    assert torch.equal(got, ref)
    assert torch.equal(call(F32), got)
    assert torch.equal(call(None), ref.to(F16 if kind == "fp16" else BF16))
    # 8-bit results of the first columns, whole blocks of them
    n = N // 32 * 32
    pick = lambda t: torch.cat([t[:, :n], t[:, N:N + n]], 1).contiguous() if gated else t[:, :n].contiguous()
    w = pick(w) if isinstance(w, torch.Tensor) else D().FP8Rows(*map(pick, w))
    got = X().grouped_linear(a, w, offsets, index=index, index_div=2, bias=pick(bias), gated=gated, out_dtype="mx")
    some = slice(None, None, 5)                                # (rows of every group's tiles)
    codes, s = OD.quantize_block(ref[some, :n].cpu().numpy())
    assert torch.equal(got.codes[some].cpu(), torch.from_numpy(codes)) and torch.equal(got.scales[some].cpu(), torch.from_numpy(s))
