"""GPU tests of linear with 4-bit weights (FP4Rows) and of quantize_fp4: every code and
scale, both activations' ranges, row counts on both sides of each kernel's limits,
epilogues, strides and guards, offsets past 32 bits, streams and replays; against the
float64 oracle."""
import itertools

import numpy as np
import pytest
import torch

from oracle import dense as OD

pytestmark = pytest.mark.gpu

BF16, F16, F32, U8 = torch.bfloat16, torch.float16, torch.float32, torch.uint8
E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
TABLE = np.concatenate([E2M1, -E2M1])


def D():
    from nvfp4_w4a4_expert_amd import dense
    return dense


def rand(shape, seed, dtype=BF16, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale).to(dtype)


def f64(t):
    return t.detach().cpu().double().numpy()


def values(codes, scales, gain=None):
    """float64 values of codes [rows, K/2] and scales, without the gain where it is None."""
    c = codes.cpu().numpy()
    v = TABLE[np.stack([c & 15, c >> 4], 2).reshape(c.shape[0], -1)]
    s = scales.cpu().numpy()
    K = v.shape[1]
    if s.shape[1] * 16 == K:
        s = np.repeat(OD.e4m3_decode(s), 16, axis=1)
    else:
        s = np.repeat(np.where(s == 255, np.nan, 2.0 ** (s.astype(np.float64) - 127)), 32, axis=1)
    return v * s * (1.0 if gain is None else float(gain))


def weights(rows, K, form, seed, gain=True):
    """FP4Rows with all codes and scales about 1 / sqrt(K)."""
    g = torch.Generator().manual_seed(seed)
    codes = torch.randint(0, 256, (rows, K // 2), generator=g, dtype=U8)
    if form == "nv":
        sf = torch.randint(0x20, 0x50, (rows, K // 16), generator=g, dtype=U8)
    else:
        sf = torch.randint(123, 130, (rows, K // 32), generator=g, dtype=U8)
    s = torch.tensor([0.37 * K ** -0.5]) if gain else None
    return D().FP4Rows(codes.cuda(), sf.cuda(), None if s is None else s.cuda()), (codes, sf, s)


def check(got, a, host, form, out, bias=None, act=None, gated=False, residual=None, label=""):
    codes, sf, s = host
    # the gain multiplies the sum: one rounding, which the oracle's budget of 64 holds;
    # fp16 against "mx" adds up twice as many products
    ref, err = OD.linear(f64(a), values(codes, sf, s), None if bias is None else f64(bias), act, gated,
                         None if residual is None else f64(residual))
    if form == "mx" and a.dtype == F16:
        v = values(codes, sf, s)
        N = v.shape[0] // 2 if gated else v.shape[0]
        plain = np.abs(f64(a)) @ np.abs(v).T
        extra = f64(a).shape[1] / 32 * OD.U
        big = 1.2 * plain[:, :N]
        if gated:
            w = f64(a) @ v.T + (0 if bias is None else f64(bias))
            big = big * np.abs(w[:, N:]) + np.abs(OD.activate(w[:, :N], act)) * plain[:, N:] + big * plain[:, N:] * extra
        err = err + extra * big
    if out == "mx":
        OD.check_fp8(got.codes.cpu().numpy(), got.scales.cpu().numpy(), ref, err, label)
        return
    want = out or a.dtype
    assert got.dtype == want and got.shape == ref.shape
    OD.check_rounded(f64(got), ref, err, want, label)


def case(M, N, K, form, dtype, act=None, gated=False, bias=None, residual=None, out=None, gain=True, seed=0):
    a = rand((M, K), seed, dtype)
    rows = 2 * N if gated else N
    w, host = weights(rows, K, form, seed + 1, gain)
    b = None if bias is None else rand((rows,), seed + 2, bias, 0.5)
    r = None if residual is None else rand((M, N), seed + 3, residual, 2.0)
    got = D().linear(a.cuda(), w, bias=None if b is None else b.cuda(), act=act, gated=gated,
                     residual=None if r is None else r.cuda(), out_dtype=out)
    check(got, a, host, form, out, b, act, gated, r, f"{M}x{N}x{K} {form} {dtype} {act} gated={gated} {out}")


FORMS = ["nv", "mx"]
TYPES = [BF16, F16]


@pytest.mark.parametrize("M", [1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 129, 200, 300])
@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("dtype", TYPES)
def test_rows_and_widths(M, form, dtype):
    for N, K in ((1, 32), (31, 96), (64, 128), (97, 416), (130, 2112)):
        case(M, N, K, form, dtype, seed=M + N)


@pytest.mark.parametrize("K", [32, 64, 160, 480, 544, 1056, 2816, 8192])
@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("dtype", TYPES)
def test_depths(K, form, dtype):
    for M in (1, 3, 20, 40, 70):
        case(M, 33, K, form, dtype, seed=K, gain=M != 3)
        case(M, 18, K, form, dtype, gated=True, act="silu", out=F32, seed=K + 1)


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("out", [BF16, F16, F32, "mx"])
@pytest.mark.parametrize("gated", [False, True])
def test_outputs(form, dtype, out, gated):
    acts = itertools.cycle([None, "silu", "gelu", "gelu_tanh", "relu"])
    for i, (M, N) in enumerate(((1, 32), (16, 96), (25, 64), (50, 224), (80, 160), (300, 352))):
        case(M, N, 224, form, dtype, next(acts), gated, [None, F32, BF16, F16][i % 4], [None, BF16, F32, F16][(i + gated) % 4], out, seed=i)


@pytest.mark.parametrize("M", [32, 96])
@pytest.mark.parametrize("dtype", TYPES)
def test_every_code_and_scale_is_exact(M, dtype):
    """Rows of a that pick one element each: the result is w's transpose, exactly."""
    for form in FORMS:
        N, K = 256, 32
        codes = torch.from_numpy(np.random.default_rng(1).integers(0, 256, (N, K // 2)).astype(np.uint8))
        codes[:, :8] = torch.tensor([0x10, 0x32, 0x54, 0x76, 0x98, 0xBA, 0xDC, 0xFE], dtype=U8)
        sf = torch.arange(256, dtype=torch.int32).to(U8)[:, None].repeat(1, 2 if form == "nv" else 1)
        a = torch.zeros(M, K, dtype=dtype)
        a[torch.arange(M), torch.arange(M) % K] = 1.0
        w = D().FP4Rows(codes.cuda(), sf.cuda())
        got = f64(D().linear(a.cuda(), w, out_dtype=F32))
        ref = values(codes, sf)
        if form == "mx":
            # 2^127 times more than 1.5 is infinite in bf16; a NaN or infinity meets the zeros of a
            ref = np.where(np.abs(ref) >= 2.0 ** 128, np.copysign(np.inf, ref), ref)
        ref = ref[:, np.arange(M) % K].T
        whole = np.isfinite(values(codes, sf)).all(1) & (np.abs(values(codes, sf)) < 2.0 ** 128).all(1)
        assert np.array_equal(got[:, whole], ref[:, whole]), form
        assert np.isnan(got[:, ~whole]).all() and (~whole).sum() == (2 if form == "nv" else 3)
        assert np.array_equal(f64(w.dequantize())[whole], values(codes, sf)[whole])


@pytest.mark.parametrize("M", [1, 20, 64, 100])
@pytest.mark.parametrize("form", FORMS)
def test_fp16_activations_over_their_whole_range(M, form):
    bits = torch.randint(-2 ** 15, 2 ** 15, (M, 352), generator=torch.Generator().manual_seed(M), dtype=torch.int32).to(torch.int16)
    a = bits.view(F16)
    a = torch.where(a.isfinite(), a, torch.zeros_like(a))
    w, host = weights(70, 352, form, 3)
    check(D().linear(a.cuda(), w, out_dtype=F32), a, host, form, F32, label=f"range {M}")
    a[0, 5], a[M - 1, 7] = float("inf"), float("nan") if M > 1 else float("inf")
    got = D().linear(a.cuda(), w, out_dtype=F32).cpu()
    assert not got[0].isfinite().any() and not got[M - 1].isfinite().any()
    codes, sf, _ = host
    v = values(codes, sf)
    if M > 1:
        assert got[M - 1].isnan().all()
        plain = torch.from_numpy(v[:, 5] != 0)
        assert torch.equal(got[0][plain], torch.where(torch.from_numpy(v[:, 5] > 0), float("inf"), -float("inf"))[plain].float())
        keep = [i for i in range(M) if i not in (0, M - 1)]
        check(D().linear(a[keep].contiguous().cuda(), w, out_dtype=F32), a[keep], host, form, F32, label="finite rows")
        assert got[keep].isfinite().all()


def test_gains():
    a = rand((5, 64), 1)
    w, (codes, sf, _) = weights(40, 64, "nv", 2, gain=False)
    for M in (5, 90):
        a = rand((M, 64), 1)
        one = D().linear(a.cuda(), w, out_dtype=F32)
        for s in (1.0, -0.5, 0.0, 2.0 ** 60, 1e-30):
            g = torch.tensor([s], device="cuda")
            assert torch.equal(D().linear(a.cuda(), D().FP4Rows(*w[:2], g), out_dtype=F32), one * s)
            assert torch.equal(D().linear(a.cuda(), D().FP4Rows(*w[:2], g.view(1, 1)), out_dtype=F32), one * s)
        assert D().linear(a.cuda(), D().FP4Rows(*w[:2], torch.tensor([float("nan")], device="cuda"))).isnan().all()


@pytest.mark.parametrize("M", [7, 64, 90])
@pytest.mark.parametrize("form", FORMS)
def test_strides_guards_and_residual_in_place(M, form):
    N, K = 72, 160
    for dtype in TYPES:
        w, host = weights(N, K, form, 1)
        wide = torch.randint(0, 256, (N, K // 2 + 48), dtype=U8, device="cuda")
        wide[:, 16:16 + K // 2] = w.codes
        ws = D().FP4Rows(wide[:, 16:16 + K // 2], w.scales, w.scale)
        ab = rand((M, K + 24), 2, dtype).cuda()
        a = ab[:, 8:8 + K]
        buf = rand((M + 2, N + 10), 3, dtype).cuda()
        r = buf[1:M + 1, 5:5 + N]
        ref = D().linear(a.contiguous(), w, residual=r.contiguous(), act="gelu")
        check(ref, a, host, form, dtype, act="gelu", residual=r, label="strides")
        keep = buf.clone()
        assert D().linear(a, ws, residual=r, act="gelu", out=r) is r
        assert torch.equal(r, ref)
        buf[1:M + 1, 5:5 + N] = keep[1:M + 1, 5:5 + N]
        assert torch.equal(buf, keep)


@pytest.mark.parametrize("M", [3, 70])
def test_offsets_past_32_bits(M):
    N, K = 600, 64
    ld = 1 << 23                                               # bytes between rows of w
    cb = torch.zeros((N - 1) * ld + K // 2, dtype=U8, device="cuda")
    w, host = weights(N, K, "nv", 1)
    codes = torch.as_strided(cb, (N, K // 2), (ld, 1))
    codes.copy_(w.codes)
    a = rand((M, K), 2)
    ob = torch.zeros((M - 1) * (1 << 26) + N, dtype=BF16, device="cuda")
    out = torch.as_strided(ob, (M, N), (1 << 26, 1))
    got = D().linear(a.cuda(), D().FP4Rows(codes, w.scales, w.scale), out=out)
    check(got, a, host, "nv", BF16, label="far rows")


def test_empty_results():
    w, _ = weights(40, 64, "nv", 1)
    assert D().linear(rand((0, 64), 1).cuda(), w).shape == (0, 40)
    none = D().FP4Rows(w.codes[:0], w.scales[:0], w.scale)
    assert D().linear(rand((9, 64), 1).cuda(), none).shape == (9, 0)


@pytest.mark.parametrize("M", [1, 40, 100])
@pytest.mark.parametrize("form,dtype", [("nv", BF16), ("mx", F16)])
def test_streams_replays_and_repeats(M, form, dtype):
    N, K = 96, 704
    w, _ = weights(2 * N, K, form, 1)
    a = rand((M, K), 2, dtype).cuda()
    call = lambda s=None: D().linear(a, w, act="silu", gated=True, out_dtype="mx", stream=s)
    ref = call()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got, raw = call(side), call(side.cuda_stream)
    side.synchronize()
    for q in (got, raw):
        assert torch.equal(q.codes, ref.codes) and torch.equal(q.scales, ref.scales)
    one, two = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()  # (each holds a workspace of its own)
    with torch.cuda.graph(one):
        got = call()
    with torch.cuda.graph(two):
        other = call()
    for s in range(3):
        a.copy_(rand((M, K), 10 + s, dtype))
        one.replay()
        two.replay()
        torch.cuda.synchronize()
        ref = call()
        for q in (got, other):
            assert torch.equal(q.codes, ref.codes) and torch.equal(q.scales, ref.scales)


@pytest.mark.parametrize("N,K", [(1, 32), (33, 96), (96, 704), (300, 2816)])
def test_quantize(N, K):
    from nvfp4_w4a4_expert_amd import moe
    w = rand((N, K), N, BF16, 0.05).cuda()
    q = D().quantize_fp4(w)
    codes, sf, s2 = moe.quantize_expert_weights(w[None].contiguous())
    assert torch.equal(q.codes, codes[0]) and torch.equal(q.scales, sf[0]) and torch.equal(q.scale, s2)
    # E2M1's half step is a sixth of the value at most, or a quarter of the scale
    amax = w.float().view(N, -1, 16).abs().amax(2).repeat_interleave(16, 1)
    assert ((q.dequantize() - w.float()).abs() <= amax * 0.19).all()
    m = D().quantize_fp4(w, "mx")
    assert m.scale is None and m.scales.shape == (N, K // 32)
    amax = w.float().view(N, -1, 32).abs().amax(2).repeat_interleave(32, 1)
    assert ((m.dequantize() - w.float()).abs() <= amax * 0.34).all()
    x = rand((4, K), 2).cuda()
    for f in (q, m):
        ref = x.double() @ f.dequantize().double().t()
        got = D().linear(x, f, out_dtype=F32)
        assert (got - ref).abs().max() < 1e-4 * ref.abs().max() + 1e-6
    pad = torch.zeros(N, K + 16, dtype=BF16, device="cuda")
    pad[:, 8:8 + K] = w
    assert torch.equal(D().quantize_fp4(pad[:, 8:8 + K]).codes, q.codes)


def test_quantize_of_zeros_and_tiny_weights():
    z = D().quantize_fp4(torch.zeros(4, 64, dtype=BF16, device="cuda"))
    assert float(z.scale) == 1.0 and not z.dequantize().any()
    for mag in (2.0 ** -120, 2.0 ** 100):
        w = (rand((8, 64), 1, F32) * mag).to(BF16).cuda()
        q = D().quantize_fp4(w)
        assert ((q.dequantize().double() - w.double()).abs() <= w.double().abs().view(8, -1, 16).amax(2).repeat_interleave(16, 1) * 0.19).all()


def test_in_a_feed_forward_with_block_norm():
    """A decoder's dense half with 4-bit weights between two norms, as it would be used."""
    T, H, I = 20, 256, 160
    x, r = rand((T, H), 1).cuda(), rand((T, H), 2).cuda()
    w_gu, w_dn = D().quantize_fp4(rand((2 * I, H), 3, BF16, 0.06).cuda()), D().quantize_fp4(rand((H, I), 4, BF16, 0.08).cuda(), "mx")
    g1, g2 = rand((H,), 5, BF16, 0.2).cuda(), rand((H,), 6, BF16, 0.2).cuda()
    n = D().block_norm(x, r, post_weight=g1, weight=g2, weight_offset=1.0, residual_scale=0.5)
    h = D().linear(n.y, w_gu, act="gelu_tanh", gated=True)
    y = D().linear(h, w_dn)
    out = D().block_norm(y, n.total, post_weight=g2, gate=0.7, weight=g1, weight_offset=1.0, scales="mx")
    t, err = OD.block_total(f64(x), f64(r), True, f64(g1), 1e-6, 1.0, 1.0, None, 0.5)
    OD.check_rounded(f64(n.total), t, err, BF16, "total")
    ref, err = OD.linear(f64(n.y), f64(w_gu.dequantize()), None, "gelu_tanh", True)
    OD.check_rounded(f64(h), ref, err + np.abs(ref) * 4 * OD.U, BF16, "gate/up")
    ref, err = OD.linear(f64(h), f64(w_dn.dequantize()))
    OD.check_rounded(f64(y), ref, err, BF16, "down")
    t, err = OD.block_total(f64(y), f64(n.total), True, f64(g2), 1e-6, 1.0, 0.7, None, 1.0)
    OD.check_rounded(f64(out.total), t, err, BF16, "total 2")
