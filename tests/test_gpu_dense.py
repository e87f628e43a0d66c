"""GPU tests of the dense operators (rms_norm, quantize_fp8, linear) against
the float64 oracle, with tolerances derived there; bit-exact for the quantiser.
Covered besides the values: strides and guards, NaN and infinities, offsets past
32 bits, streams, graph replays, and the operators around a routed-expert layer."""
import itertools

import numpy as np
import pytest
import torch

from oracle import dense as OD

pytestmark = pytest.mark.gpu

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32


def D():
    from nvfp4_w4a4_expert_amd import dense
    return dense


def rand(shape, seed, dtype=BF16, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale).to(dtype)


def f64(t):
    return t.detach().cpu().double().numpy()


def f32(t):
    return t.detach().cpu().float().numpy()


def fp8_np(r):
    return r.codes.cpu().numpy(), r.scales.cpu().numpy()


# ---- rms_norm ------------------------------------------------------------------

def norm_case(T, K, dtype, residual, weight, offset, scales, want_y=True, seed=0, eps=1e-6):
    x = rand((T, K), seed, dtype)
    x[:, :: max(1, K // 5)] *= 20
    r = rand((T, K), seed + 1, dtype, 3.0) if residual else None
    w = rand((K,), seed + 2, dtype, 0.3) if weight else None
    n = D().rms_norm(x.cuda(), None if w is None else w.cuda(), residual=None if r is None else r.cuda(),
                     eps=eps, weight_offset=offset, want_y=want_y, scales=scales)
    s = x if r is None else (x.float() + r.float()).to(dtype)
    if r is not None:
        assert torch.equal(n.total.cpu(), s)
    y, err = OD.rms_norm(f64(s), None if w is None else f64(w), eps, offset)
    label = f"{T}x{K} {dtype} {scales}"
    if want_y:
        OD.check_rounded(f64(n.y), y, err, dtype, label)
    else:
        assert n.y is None
    if scales:
        OD.check_fp8(*fp8_np(n.fp8), y, err, label)


# each thread-group width of the kernel, whole and ragged, and its edges
WIDTHS = [8, 24, 128, 136, 256, 264, 504, 512, 520, 1024, 1032, 2048, 2056, 2816, 4096, 4104, 8192, 8200, 16384, 16392, 32768]


@pytest.mark.parametrize("K", WIDTHS)
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_norm_widths(K, dtype):
    for T, scales in ((1, "row"), (5, None), (18, "row")):
        norm_case(T, K, dtype, T != 5, True, 1.0, scales, seed=K + T)
    if K % 32 == 0:
        norm_case(7, K, dtype, True, True, 0.0, "mx", seed=K)


@pytest.mark.parametrize("residual,weight,scales,want_y", [
    c for c in itertools.product([False, True], [False, True], [None, "row", "mx"], [False, True])
    if c[0] or c[2] or c[3]])
def test_norm_outputs(residual, weight, scales, want_y):
    norm_case(9, 704, BF16, residual, weight, 0.5, scales, want_y, seed=3)
    norm_case(3, 2816, F16, residual, weight, 0.0, scales, want_y, seed=4)


def test_norm_eps_and_zero_rows():
    x = torch.zeros(6, 96, dtype=BF16)
    x[1] = 1.0
    x[2, 5] = 2.0 ** -60
    x[4] = 2.0 ** -70
    for eps in (0.0, 1e-6, 2.5):
        rows = [1, 2, 4] if eps == 0 else list(range(6))     # 0 / sqrt(0) has no value
        n = D().rms_norm(x[rows].contiguous().cuda(), eps=eps, scales="row")
        m = D().rms_norm(x[rows].contiguous().cuda(), eps=eps, scales="mx")
        s = f64(x[rows])
        y = s / np.sqrt((s * s).mean(1, keepdims=True) + eps)
        if eps == 0:
            # squares of 2^-70 and 2^-60 are normal fp32 numbers: the norm is exact to rounding
            OD.check_rounded(f64(n.y), y, np.abs(y) * 36 * OD.U, BF16)
        else:
            OD.check_rounded(f64(n.y), y, np.abs(y) * 36 * OD.U + 2.0 ** -148, BF16)
            assert fp8_np(n.fp8)[1][0] == 0 and not fp8_np(n.fp8)[0][0].any()
            assert not fp8_np(m.fp8)[0][0].any() and np.all(fp8_np(m.fp8)[1][0] == 1)
        OD.check_fp8(*fp8_np(m.fp8), y, np.abs(y) * 36 * OD.U + 2.0 ** -148)


def test_norm_nan_and_inf_stay_in_their_rows():
    x = rand((5, 256), 1)
    x[1, 7] = float("nan")
    x[3, 9] = float("-inf")
    for scales in ("row", "mx"):
        n = D().rms_norm(x.cuda(), scales=scales)
        y = n.y.cpu().float()
        assert y[1].isnan().all() and y[3, 9].isnan()
        assert (y[3, torch.arange(256) != 9] == 0).all()
        codes, _ = fp8_np(n.fp8)
        assert np.all((codes[1] & 0x7F) == 0x7F) and (codes[3, 9] & 0x7F) == 0x7F
        assert not (np.delete(codes[3], 9) & 0x7F).any()
        good = [0, 2, 4]
        ref, err = OD.rms_norm(f64(x)[good], None, 1e-6, 0.0)
        OD.check_rounded(f64(n.y)[good], ref, err, BF16)


def test_norm_strided_in_place_and_guarded():
    T, K = 11, 264
    wide = rand((T + 2, 2 * K + 16), 5).cuda()
    x, r = wide[1:T + 1, 8:8 + K], wide[1:T + 1, 8 + K:8 + 2 * K]
    before = wide.clone()
    s = (x.float() + r.float()).to(BF16)
    y, err = OD.rms_norm(f64(s), None, 1e-5, 0.0)
    # the residual stream updated in place, y into x itself
    n = D().rms_norm(x, residual=r, eps=1e-5, total_out=r, out=x, scales="row")
    assert n.y is x and n.total is r and torch.equal(r, s)
    OD.check_rounded(f64(x), y, err, BF16)
    OD.check_fp8(*fp8_np(n.fp8), y, err)
    keep = torch.ones_like(wide, dtype=torch.bool)
    keep[1:T + 1, 8:8 + 2 * K] = False
    assert torch.equal(wide[keep], before[keep])


def test_norm_total_into_x_and_empty():
    x, r = rand((4, 128), 6).cuda(), rand((4, 128), 7).cuda()
    s = (x.float() + r.float()).to(BF16)
    n = D().rms_norm(x, residual=r, total_out=x, want_y=False)
    assert n.total is x and torch.equal(x, s) and n.y is None and n.fp8 is None
    n = D().rms_norm(x[:0], residual=r[:0], scales="mx")
    assert n.y.shape == (0, 128) and n.fp8.codes.shape == (0, 128) and n.fp8.scales.shape == (0, 4)


# ---- quantize_fp8 ----------------------------------------------------------------

def quant_rows(T, K, dtype, seed):
    x = rand((T, K), seed, dtype)
    x[:, ::7] *= 30
    flat = x.view(-1)
    special = torch.tensor([0.0, -0.0, 448.0, -448.0, 447.9, 464.0, 2.0 ** -9, 2.0 ** -10, 3 * 2.0 ** -10, 57344.0,
                            float("inf"), float("-inf"), float("nan"), 2.0 ** -14, 6e-8, 1.0, 1.75, 0.875, 1.0625])
    at = torch.randperm(flat.numel(), generator=torch.Generator().manual_seed(seed))[:special.numel()]
    flat[at] = special[:at.numel()].to(dtype)
    if T > 2:
        x[1] = 0
        x[2] *= 2.0 ** (-120 if dtype == BF16 else -12)      # scales at the bottom of their range
    if T > 4 and dtype == BF16:
        x[3] *= 2.0 ** 120                                   # and near the top
        x[4] = 2.0 ** -133                                   # fp32 subnormals
    return x


@pytest.mark.parametrize("K", WIDTHS)
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_quantize_is_exact(K, dtype):
    for T in (1, 6, 19):
        x = quant_rows(T, K, dtype, K + T)
        c, s = fp8_np(D().quantize_fp8(x.cuda(), "row"))
        rc, rs = OD.quantize_row(f32(x))
        assert np.array_equal(s.view(np.uint32), rs.view(np.uint32))
        nan = (rc & 0x7F) == 0x7F
        assert np.array_equal(np.where(nan, 0x7F, rc), np.where((c & 0x7F) == 0x7F, 0x7F, c))
        if K % 32 == 0:
            c, s = fp8_np(D().quantize_fp8(x.cuda(), "mx"))
            rc, rs = OD.quantize_block(f32(x))
            assert np.array_equal(s, rs)
            assert np.array_equal(np.where((rc & 0x7F) == 0x7F, 0x7F, rc), np.where((c & 0x7F) == 0x7F, 0x7F, c))


def test_quantize_every_bf16_value():
    """All 65536 bf16 patterns, one per block of 32 with a fixed companion, and in
    one row each of 8."""
    bits = np.arange(65536, dtype=np.uint16)
    x = torch.from_numpy(bits.view(np.int16).copy()).view(BF16)
    b = torch.zeros(2048, 32 * 32, dtype=BF16)
    b.view(-1)[::32] = x
    b.view(-1)[5::32] = 1.0
    c, s = fp8_np(D().quantize_fp8(b.cuda(), "mx"))
    rc, rs = OD.quantize_block(f32(b))
    assert np.array_equal(s, rs) and np.array_equal(rc & 0x7F, c & 0x7F)
    r = torch.zeros(65536, 8, dtype=BF16)
    r[:, 3] = x
    c, s = fp8_np(D().quantize_fp8(r.cuda(), "row"))
    rc, rs = OD.quantize_row(f32(r))
    assert np.array_equal(s.view(np.uint32), rs.view(np.uint32)) and np.array_equal(rc & 0x7F, c & 0x7F)


def test_quantize_strided_and_dequantize():
    x = rand((40, 200), 8).cuda()
    v = x[::2, 8:104]
    q = D().quantize_fp8(v, "mx")
    rc, rs = OD.quantize_block(f32(v))
    assert np.array_equal(q.codes.cpu().numpy(), rc) and np.array_equal(q.scales.cpu().numpy(), rs)
    assert np.array_equal(f64(q.dequantize()), OD.dequantize(rc, rs))
    q = D().quantize_fp8(v, "row")
    assert np.allclose(f64(q.dequantize()), OD.dequantize(*OD.quantize_row(f32(v))), rtol=2 ** -23, atol=0)


# ---- linear ----------------------------------------------------------------------

def operand(shape, seed, kind, scale):
    """(device operand, float64 values)."""
    if kind in ("bf16", "fp16"):
        t = rand(shape, seed, BF16 if kind == "bf16" else F16, scale)
        return t.cuda(), f64(t)
    t = rand(shape, seed, F32, scale).numpy()
    codes, scales = OD.quantize_row(t) if kind == "row" else OD.quantize_block(t)
    return D().FP8Rows(torch.from_numpy(codes).cuda(), torch.from_numpy(scales).cuda()), OD.dequantize(codes, scales)


def scaled(kind, out):
    """Whether linear may run the scaled 8-bit instruction: wherever the output is
    16 bits wide."""
    return kind in ("row", "mx") and out in (None, BF16, F16)


def linear_case(M, N, K, kind, act=None, gated=False, bias=None, residual=None, out=None, seed=0):
    a, av = operand((M, K), seed, kind, 1.0)
    rows = 2 * N if gated else N
    w, wv = operand((rows, K), seed + 1, kind, K ** -0.5)
    b = None if bias is None else rand((rows,), seed + 2, bias, 0.5)
    r = None if residual is None else rand((M, N), seed + 3, residual, 2.0)
    got = D().linear(a, w, bias=None if b is None else b.cuda(), act=act, gated=gated,
                     residual=None if r is None else r.cuda(), out_dtype=out)
    ref, err = OD.linear(av, wv, None if b is None else f64(b), act, gated, None if r is None else f64(r),
                         scaled(kind, out))
    label = f"{M}x{N}x{K} {kind} {act} gated={gated} out={out}"
    if out == "mx":
        OD.check_fp8(*fp8_np(got), ref, err, label)
        return
    want = out or (F16 if kind == "fp16" else BF16)
    assert got.dtype == want and got.shape == (M, N)
    OD.check_rounded(f64(got), ref, err, want, label)


KINDS = ["bf16", "fp16", "row", "mx"]
# few rows, their edges, each tile size, ragged in every direction
ROWS = [1, 2, 15, 16, 17, 33, 64, 65, 127, 200]


@pytest.mark.parametrize("M", ROWS)
@pytest.mark.parametrize("kind", KINDS)
def test_linear_rows_and_widths(M, kind):
    for N, K in ((1, 32), (31, 96), (64, 128), (97, 416), (130, 2112)):
        linear_case(M, N, K, kind, seed=M + N)


@pytest.mark.parametrize("kind,K", [("bf16", 8), ("bf16", 56), ("bf16", 72), ("fp16", 200), ("row", 16), ("row", 112), ("row", 144),
                                    ("mx", 32), ("mx", 160), ("mx", 544)])
def test_linear_short_and_ragged_depths(kind, K):
    for M, N in ((3, 33), (40, 18), (90, 70), (260, 300)):
        linear_case(M, N, K, kind, seed=K)
        linear_case(M, N, K, kind, gated=True, act="silu", out=F32, seed=K + 1)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("out", [BF16, F16, F32, "mx"])
@pytest.mark.parametrize("gated", [False, True])
def test_linear_outputs(kind, out, gated):
    acts = itertools.cycle([None, "silu", "gelu", "gelu_tanh", "relu"])
    for i, (M, N) in enumerate(((1, 32), (16, 96), (50, 224), (80, 160), (300, 352))):
        linear_case(M, N, 224, kind, next(acts), gated, [None, F32, BF16, F16][i % 4], [None, BF16, F32, F16][(i + gated) % 4], out,
                    seed=i + 10 * gated)


@pytest.mark.parametrize("act", [None, "none", "silu", "gelu", "gelu_tanh", "relu"])
@pytest.mark.parametrize("gated", [False, True])
def test_linear_activations(act, gated):
    for M in (4, 130):
        linear_case(M, 65, 64, "bf16", act, gated, F32, None, F32, seed=M)


def test_activation_range():
    """Every activation over large and small arguments: a 1 x 1 weight passes v
    itself (K = 8, the other elements 0), so out is act(v) to rounding."""
    v = np.concatenate([-np.logspace(-30, 30, 400), [0.0], np.logspace(-30, 30, 400), np.linspace(-12, 12, 1001)])
    a = torch.zeros(v.size, 8, dtype=BF16)
    a[:, 0] = torch.from_numpy(v).to(BF16)
    w = torch.zeros(1, 8, dtype=BF16)
    w[0, 0] = 1.0
    x = f64(a)[:, :1]
    for act in ("silu", "gelu", "gelu_tanh", "relu"):
        got = f64(D().linear(a.cuda(), w.cuda(), act=act, out_dtype=F32))
        ref = OD.activate(x, act)
        # relative: the exponent's argument z is rounded (|z| u of the result, z <= 100 where it
        # has not underflowed: z = v, 2u <= 2.3 v^2 u relative...), erfc's fit 1.2e-7
        z = np.minimum(np.abs(x) if act == "silu" else 2.4 * np.abs(x) + 0.1 * np.abs(x) ** 3 if act == "gelu_tanh"
                       else x * x, 110.0)
        tol = np.abs(ref) * (8 * z + 24) * OD.U + 2.0 ** -126
        assert np.all(np.abs(got - ref) <= tol), act


@pytest.mark.parametrize("M,N,K,kind,gated,out", [
    (300, 1411, 704, "fp16", False, F16), (520, 2112, 704, "mx", True, "mx"), (1030, 2816, 416, "bf16", False, BF16),
    (2050, 2100, 136, "bf16", True, BF16), (2050, 4200, 160, "row", False, F32), (4100, 3100, 96, "mx", False, BF16),
    (2500, 2560, 64, "mx", True, "mx"), (4096, 128, 2816, "bf16", False, F32)])
def test_linear_large(M, N, K, kind, gated, out):
    linear_case(M, N, K, kind, "gelu_tanh" if gated else None, gated, F32, None if out == "mx" else BF16, out, seed=M)


def workspace(M, N, K, kind, out, gated):
    from nvfp4_w4a4_expert_amd import _lib as L
    types = {"bf16": L.TYPE_BF16, "fp16": L.TYPE_FP16, "row": L.TYPE_FP8_ROW, "mx": L.TYPE_FP8_MX}
    outs = {BF16: L.TYPE_BF16, F16: L.TYPE_FP16, F32: L.TYPE_FP32, "mx": L.TYPE_FP8_MX}
    return L.linear_workspace_size(L.Linear(M=M, N=N, K=K, type=types[kind], out_type=outs[out], gated=gated))


# sizes whose last round is cut along K: all of the tiles or the last ones, parts of
# equal and of unequal length, a ragged last step, every kind of output
@pytest.mark.parametrize("M,N,K,kind,gated,out", [
    (17, 130, 2816, "bf16", False, F32), (17, 31, 2808, "fp16", True, F16), (48, 128, 2816, "bf16", False, F32),
    (40, 96, 2848, "mx", True, "mx"), (64, 320, 5632, "mx", False, BF16), (33, 77, 2832, "row", False, F32),
    (65, 128, 4224, "row", False, "mx"), (300, 127, 2816, "bf16", True, BF16), (130, 64, 8192, "mx", False, F32),
    (2300, 130, 2112, "bf16", False, BF16), (4100, 2112, 1416, "bf16", True, BF16), (4096, 2112, 2816, "mx", True, "mx")])
def test_linear_cut_along_k(M, N, K, kind, gated, out):
    assert workspace(M, N, K, kind, out, gated) > 0
    linear_case(M, N, K, kind, "gelu_tanh" if gated else "silu", gated, BF16, F32 if out == F32 else BF16, out, seed=N)


@pytest.mark.parametrize("M", [3, 40, 100, 300])
@pytest.mark.parametrize("kind", KINDS)
def test_linear_strides_edges_and_guards(M, kind):
    """Operands and result are column ranges of wider buffers filled with NaN
    (codes 0x7F): nothing outside is read into a result or written."""
    N, K = 77, 96
    dt = {"bf16": BF16, "fp16": F16}.get(kind)
    vals = {}

    def strided(rows, seed, scale):
        t, v = operand((rows, K), seed, kind, scale)
        src = t if dt is not None else t.codes
        wide = torch.full((rows + 3, K + 160), float("nan"), dtype=dt, device="cuda") if dt is not None else \
            torch.full((rows + 3, K + 160), 0x7F, dtype=torch.uint8, device="cuda")
        view = wide[1:rows + 1, 64:64 + K]
        view.copy_(src)
        vals[seed] = v
        return view if dt is not None else D().FP8Rows(view, t.scales)

    a, w = strided(M, 21, 1.0), strided(N, 22, 0.1)
    r = rand((M, N), 23)
    buf = torch.full((M + 2, N + 11), 7.0, dtype=BF16, device="cuda")
    out = buf[1:M + 1, 5:5 + N]
    out.copy_(r)
    keep = torch.ones_like(buf, dtype=torch.bool)
    keep[1:M + 1, 5:5 + N] = False
    got = D().linear(a, w, residual=out, out=out)                 # in place over the residual
    assert got is out
    ref, err = OD.linear(vals[21], vals[22], residual=f64(r), scaled=scaled(kind, BF16))
    OD.check_rounded(f64(out), ref, err, BF16)
    assert (buf[keep] == 7.0).all()


@pytest.mark.parametrize("kind", ["bf16", "row", "mx"])
def test_linear_nan_and_inf_stay_in_their_rows(kind):
    for M in (7, 120):
        a, av = operand((M, 160), 31, kind, 1.0)
        w, wv = operand((50, 160), 32, kind, 0.1)
        if kind == "bf16":
            a[2, 11] = float("nan")
            a[5, 3] = float("inf")
        else:
            a.codes[2, 11] = 0x7F
            a.codes[5, 3] = 0xFF
        got = D().linear(a, w, out_dtype=F32).cpu()
        bad = torch.zeros(M, dtype=torch.bool)
        bad[[2, 5]] = True
        assert got[2].isnan().all() and not got[5].isfinite().any() and got[~bad].isfinite().all()
        ref, err = OD.linear(av, wv)
        OD.check_rounded(f64(got)[~bad.numpy()], ref[~bad.numpy()], err[~bad.numpy()], F32)


@pytest.mark.parametrize("M", [5, 40, 300])
@pytest.mark.parametrize("ca,cw", [(1, 127), (3, 240), (7, 247), (240, 3), (127, 127)])
def test_linear_block_scale_range(M, ca, cw):
    """Scale codes towards the ends of their range.  Elements (2^-3 to 7.5) times
    scales are normal numbers or multiples of 2^-133; other rows' scales of a
    make the products' scale 1."""
    g = torch.Generator().manual_seed(M + ca)
    rows = lambda n: (torch.randint(0x20, 0x50, (n, 256), generator=g) +
                      128 * torch.randint(0, 2, (n, 256), generator=g)).to(torch.uint8)
    a, w = rows(M), rows(64)
    sa = torch.full((M, 8), 254 - cw, dtype=torch.uint8)
    sa[::2] = ca
    sw = torch.full((64, 8), cw, dtype=torch.uint8)
    av, wv = (OD.dequantize(c.numpy(), s.numpy()) for c, s in ((a, sa), (w, sw)))
    for out in (F32, BF16):
        ref, err = OD.linear(av, wv, scaled=scaled("mx", out))
        got = D().linear(D().FP8Rows(a.cuda(), sa.cuda()), D().FP8Rows(w.cuda(), sw.cuda()), out_dtype=out)
        OD.check_rounded(f64(got), ref, err, out)


@pytest.mark.parametrize("M,N,K,gated", [(1, 32, 64, False), (9, 96, 128, True), (70, 160, 256, False), (300, 256, 192, True),
                                         (260, 2112, 1024, True), (4096, 128, 2816, False)])
@pytest.mark.parametrize("kind", ["bf16", "row", "mx"])
def test_linear_mx_is_fp32_result_quantized(M, N, K, gated, kind):
    """The 8-bit result is the quantiser's form of the fp32 one, code for code (both
    run the same products and epilogue), with infinities, NaN and zero blocks among
    the results."""
    a, _ = operand((M, K), 90 + M, kind, 1.0)
    w, _ = operand((2 * N if gated else N, K), 91 + N, kind, K ** -0.5)
    b = rand((2 * N if gated else N,), 92, F32)
    b[3], b[9], b[N // 2] = float("inf"), float("-inf"), float("nan")
    r = rand((M, N), 93, F32)
    r[M // 2, ::5] *= 2.0 ** 60
    r[M // 3, 1] = float("nan")
    kw = dict(bias=b.cuda(), gated=gated, act="relu" if gated else None, residual=r.cuda())
    want = D().linear(a, w, out_dtype=F32, **kw)
    got = D().linear(a, w, out_dtype="mx", **kw)
    rc, rs = OD.quantize_block(f32(want))
    c, s = fp8_np(got)
    assert np.array_equal(s, rs)
    nan = (rc & 0x7F) == 0x7F
    assert nan.any() and np.array_equal(nan, (c & 0x7F) == 0x7F) and np.array_equal(rc[~nan], c[~nan])


def test_offsets_past_32_bits():
    """Rows beyond 2^31 elements and 2^32 bytes of an operand, the residual and the
    result: the last rows are those of a call on them alone."""
    M, N, K = 70100, 32768, 64
    a, w = rand((M, K), 35).cuda(), rand((N, K), 36, scale=0.1).cuda()
    res = torch.ones((M, N), dtype=BF16, device="cuda")
    got = D().linear(a, w, residual=res, out=res)
    for lo, hi in ((0, 300), (M - 300, M)):
        ref, err = OD.linear(f64(a[lo:hi]), f64(w[:512]), residual=1.0)
        OD.check_rounded(f64(got[lo:hi, :512]), ref, err, BF16)
        ref, err = OD.linear(f64(a[lo:hi]), f64(w[-512:]), residual=1.0)
        OD.check_rounded(f64(got[lo:hi, -512:]), ref, err, BF16)
    # the same buffer as norm input, in place, and as an operand of many rows
    tail = got[-3:].clone()
    n = D().rms_norm(got, out=got, scales="mx")
    y, err = OD.rms_norm(f64(tail), None, 1e-6, 0.0)
    OD.check_rounded(f64(got[-3:]), y, err, BF16)
    OD.check_fp8(n.fp8.codes[-3:].cpu().numpy(), n.fp8.scales[-3:].cpu().numpy(), y, err)
    out = D().linear(got, rand((16, N), 37, scale=0.01).cuda(), out_dtype=F32)
    ref, err = OD.linear(f64(got[-3:]), f64(rand((16, N), 37, scale=0.01)))
    OD.check_rounded(f64(out[-3:]), ref, err, F32)


def test_linear_empty():
    w = rand((24, 64), 41).cuda()
    assert D().linear(rand((0, 64), 40).cuda(), w).shape == (0, 24)
    assert D().linear(rand((5, 64), 40).cuda(), w[:0]).shape == (5, 0)
    q = D().linear(rand((0, 64), 40).cuda(), rand((64, 64), 42).cuda(), out_dtype="mx")
    assert q.codes.shape == (0, 64) and q.scales.shape == (0, 2)


# ---- streams, graphs, determinism ---------------------------------------------------

def chain(x, h, wn, wr, wgu, wd):
    n = D().rms_norm(x, wn, residual=h, weight_offset=1.0, scales="mx")
    logits = D().linear(n.y, wr, out_dtype=F32)
    a = D().linear(n.fp8, wgu, act="gelu_tanh", gated=True, out_dtype="mx")
    return n, logits, a, D().linear(a, wd, residual=n.total)


def chain_inputs(T, seed, H=256, I=160, E=24):
    x, h = rand((T, H), seed).cuda(), rand((T, H), seed + 1, scale=2.0).cuda()
    wn = rand((H,), seed + 2, scale=0.2).cuda()
    wr = rand((E, H), seed + 3, scale=H ** -0.5).cuda()
    wgu = D().quantize_fp8(rand((2 * I, H), seed + 4, scale=H ** -0.5).cuda())
    wd = D().quantize_fp8(rand((H, I), seed + 5, scale=I ** -0.5).cuda())
    return x, h, wn, wr, wgu, wd


SMALL, MODEL = dict(H=256, I=160, E=24), dict(H=2816, I=704, E=128)       # MODEL's products are cut along K


@pytest.mark.parametrize("T,sizes", [(1, SMALL), (16, SMALL), (70, SMALL), (400, SMALL), (16, MODEL), (33, MODEL), (260, MODEL)])
def test_chain_stage_by_stage(T, sizes):
    x, h, wn, wr, wgu, wd = chain_inputs(T, 50, **sizes)
    n, logits, a, out = chain(x, h, wn, wr, wgu, wd)
    s = (x.float() + h.float()).to(BF16)
    assert torch.equal(n.total, s)
    y, err = OD.rms_norm(f64(s), f64(wn), 1e-6, 1.0)
    OD.check_rounded(f64(n.y), y, err, BF16, "y")
    OD.check_fp8(*fp8_np(n.fp8), y, err, "norm")
    ref, err = OD.linear(f64(n.y), f64(wr))
    OD.check_rounded(f64(logits), ref, err, F32, "logits")
    ref, err = OD.linear(OD.dequantize(*fp8_np(n.fp8)), OD.dequantize(*fp8_np(wgu)), act="gelu_tanh", gated=True,
                         scaled=scaled("mx", "mx"))
    OD.check_fp8(*fp8_np(a), ref, err, "gate/up")
    ref, err = OD.linear(OD.dequantize(*fp8_np(a)), OD.dequantize(*fp8_np(wd)), residual=f64(n.total),
                         scaled=scaled("mx", BF16))
    OD.check_rounded(f64(out), ref, err, BF16, "down")


def same(p, q):
    return torch.equal(p[0].y, q[0].y) and torch.equal(p[0].fp8.codes, q[0].fp8.codes) and \
        torch.equal(p[0].fp8.scales, q[0].fp8.scales) and torch.equal(p[1], q[1]) and \
        torch.equal(p[2].codes, q[2].codes) and torch.equal(p[2].scales, q[2].scales) and torch.equal(p[3], q[3])


@pytest.mark.parametrize("T,sizes", [(4, SMALL), (300, SMALL), (20, MODEL), (150, MODEL)])
def test_two_streams_and_repeats(T, sizes):
    one, two = chain_inputs(T, 60, **sizes), chain_inputs(T, 70, **sizes)
    want = chain(*one), chain(*two)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    got = []
    for _ in range(4):
        with torch.cuda.stream(s1):
            p = chain(*one)
        with torch.cuda.stream(s2):
            q = chain(*two)
        got.append((p, q))
    torch.cuda.synchronize()
    for p, q in got:
        assert same(p, want[0]) and same(q, want[1])


@pytest.mark.parametrize("raw", [False, True])
def test_stream_argument(raw):
    x, w = rand((33, 128), 80).cuda(), rand((40, 128), 81).cuda()
    want = D().rms_norm(x, scales="row"), D().linear(x, w), D().quantize_fp8(x)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    arg = s.cuda_stream if raw else s
    got = D().rms_norm(x, scales="row", stream=arg), D().linear(x, w, stream=arg), D().quantize_fp8(x, stream=arg)
    s.synchronize()
    assert torch.equal(want[0].y, got[0].y) and torch.equal(want[0].fp8.codes, got[0].fp8.codes)
    assert torch.equal(want[1], got[1]) and torch.equal(want[2].codes, got[2].codes)


def test_stream_zero_and_refused_streams():
    x = rand((33, 128), 82).cuda()
    want = D().quantize_fp8(x)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):                               # not the current stream: the default one
        handle, ctx = D()._on((x,), 0)
        with ctx:
            assert handle == 0 and torch.cuda.current_stream() == torch.cuda.default_stream()
        got = D().quantize_fp8(x, stream=0)
    torch.cuda.synchronize()
    assert torch.equal(got.codes, want.codes) and torch.equal(got.scales, want.scales)
    with pytest.raises(ValueError):
        D().quantize_fp8(x, stream="default")


@pytest.mark.parametrize("T,sizes", [(3, SMALL), (290, SMALL), (20, MODEL), (150, MODEL)])
def test_graph_replays(T, sizes):
    args = chain_inputs(T, 90, **sizes)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        chain(*args)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = chain(*args)
    for k in range(5):
        fresh = chain_inputs(T, 100 + k, **sizes)
        args[0].copy_(fresh[0])
        args[1].copy_(fresh[1])
        graph.replay()
        if k % 2:
            torch.cuda.synchronize()
        assert same(chain(*args), got)


def test_two_graphs_share_nothing():
    """Two captured calls with a workspace each, replayed on two streams at once."""
    one, two = chain_inputs(20, 110, **MODEL), chain_inputs(20, 120, **MODEL)
    want = chain(*one), chain(*two)
    graphs, outs = [], []
    for args in (one, two):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(chain(*args))
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in graphs]
    for _ in range(5):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        assert same(outs[0], want[0]) and same(outs[1], want[1])


# ---- beside the routed experts --------------------------------------------------------

@pytest.mark.parametrize("T", [1, 16, 200])
def test_layer_with_routed_and_dense_halves(T):
    """A MoE layer as it runs: pre-norm with the residual, router logits by
    linear, routed experts on the norm's bf16 rows, the dense half on its 8-bit
    rows, both added to the residual stream."""
    from nvfp4_w4a4_expert_amd import _lib, moe
    H, I, E, k = 256, 128, 8, 2
    x, h, wn, wr, wgu, wd = chain_inputs(T, 130, H=H, I=I, E=E)
    w13, w13s, w13s2 = moe.quantize_expert_weights(rand((E, 2 * I, H), 140, scale=H ** -0.5).cuda())
    w2, w2s, w2s2 = moe.quantize_expert_weights(rand((E, H, I), 141, scale=I ** -0.5).cuda())
    ones = np.full(E, 4.0 / 2688, dtype=np.float32)
    layer = moe.NVFP4MoELayer(w13, w13s, w13s2, w2, w2s, w2s2, ones, ones)
    n, logits, a, out = chain(x, h, wn, wr, wgu, wd)
    got = layer.forward(n.y, logits, k, residual=out)
    # the router's ids follow the logits; the layer sees the same rows as a direct call
    ids = torch.empty(T, k, dtype=torch.int32, device="cuda")
    wts = torch.empty(T, k, dtype=torch.float32, device="cuda")
    _lib.route_topk(logits, T, E, k, ids, wts)
    ref, err = OD.linear(f64(n.y), f64(wr))
    top = np.take_along_axis(ref, ids.cpu().numpy().astype(np.int64), 1)
    rest = np.partition(ref, E - k, axis=1)[:, E - k]
    assert np.all(top.min(1) >= rest - 2 * (err.max() + OD.U * np.abs(ref).max()))
    alone = layer.forward(n.y, logits, k)
    # got = bf16(residual + sum): alone is bf16(sum), off by half a step itself
    tol = 2.0 ** -8 * (np.abs(f64(alone)) + np.abs(f64(alone)) + np.abs(f64(out)) + np.abs(f64(got))) + 2.0 ** -120
    assert np.all(np.abs(f64(got) - (f64(out) + f64(alone))) <= tol)
