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


# ---- sums of the scaled instruction ----------------------------------------------------

def cancelling(rows, K, rng, sign):
    """In each group of eight two large elements, whose products with the other
    operand's cancel exactly (sign -1 on one side), among small ones."""
    c = (rng.integers(0x20, 0x40, (rows, K)) | 128 * rng.integers(0, 2, (rows, K))).astype(np.uint8)
    big = (rng.integers(0x60, 0x7F, (rows, K // 8)) | 128 * rng.integers(0, 2, (rows, K // 8))).astype(np.uint8)
    c[:, 1::8] = big
    c[:, 5::8] = big ^ (0x80 if sign < 0 else 0)
    return c


DATA = {"random": lambda n, K, rng, s: OD.e4m3_encode(np.clip(rng.standard_normal((n, K)) * 100, -448, 448)),
        "positive": lambda n, K, rng, s: OD.e4m3_encode(np.clip(np.abs(rng.standard_normal((n, K))) * 100, 0, 448)),
        "every code": lambda n, K, rng, s: (rng.integers(0, 0x7F, (n, K)) | 128 * rng.integers(0, 2, (n, K))).astype(np.uint8),
        "cancelling": cancelling}


@pytest.mark.parametrize("M,N,K", [(17, 33, 160), (65, 96, 512), (300, 130, 1056), (1500, 2816, 544), (4096, 2816, 2112)])
@pytest.mark.parametrize("kind", ["row", "mx"])
@pytest.mark.parametrize("data", list(DATA))
def test_scaled_sums_follow_the_cut(M, N, K, kind, data):
    """16-bit results of 8-bit operands are the cut sums (OD.cut_sums) to fp32 accuracy
    and one rounding, for sums of one sign and for sums that cancel as well; on some
    rows and columns of every tile."""
    from nvfp4_w4a4_expert_amd import _lib as L
    for out, t in ((BF16, L.TYPE_BF16), (F16, L.TYPE_FP16)):
        p = L.Linear(M=M, N=N, K=K, type=L.TYPE_FP8_ROW if kind == "row" else L.TYPE_FP8_MX, out_type=t)
        assert L.linear_workspace_size(p) == 0                 # one run over K, as in cut_sums
    rng = np.random.default_rng(M + N)
    ca, cw = DATA[data](M, K, rng, 1), DATA[data](N, K, rng, -1)
    i = np.unique(np.r_[0:3, rng.integers(0, M, 40), M - 3:M])
    j = np.unique(np.r_[0:3, rng.integers(0, N, 50), N - 3:N])
    if kind == "row":
        sa, sw = (rng.uniform(0.5, 2, n).astype(np.float32) * np.float32(2.0 ** -12 / K) ** 0.5 for n in (M, N))
        sa, sw = sa.astype(np.float32), sw.astype(np.float32)
        s, err = OD.cut_sums(OD.e4m3_decode(ca[i]), OD.e4m3_decode(cw[j]))
        both = sa[i].astype(np.float64)[:, None] * sw[j].astype(np.float64)[None]
        s, err = s * both, err * both + 2 * OD.U * np.abs(s * both)
    else:
        # (down to about 1 / sqrt(K) of E4M3's size, so that fp16 holds the results)
        sa, sw = (rng.integers(119, 122, (n, K // 32)).astype(np.uint8) for n in (M, N))
        s, err = OD.cut_sums(OD.dequantize(ca[i], sa[i]), OD.dequantize(cw[j], sw[j]))
    a = D().FP8Rows(torch.from_numpy(ca).cuda(), torch.from_numpy(sa).cuda())
    w = D().FP8Rows(torch.from_numpy(cw).cuda(), torch.from_numpy(sw).cuda())
    assert np.abs(s).max() < 6e4
    for out in (BF16, F16):
        got = f64(D().linear(a, w, out_dtype=out))[np.ix_(i, j)]
        OD.check_rounded(got, s, err, out, f"{kind} {data} {out}")


# ---- activations -----------------------------------------------------------------------

@pytest.mark.parametrize("M", [1, 20])
@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
def test_activation_error(act, M):
    """act(v) for fp32 v (the bias of a product of zeros) within the half steps that
    its exponent allows (OD.activation_error), also where the result is tiny."""
    rng = np.random.default_rng(3)
    v = np.concatenate([rng.uniform(-1, 1, 3000) * s for s in (1e-3, 1, 4, 16)] +
                       [rng.uniform(-i - 1, -i, 1000) for i in range(15)] + [rng.uniform(-90, 90, 4000)]).astype(np.float32)
    a = torch.zeros(M, 8, dtype=BF16, device="cuda")
    w = torch.zeros(v.size, 8, dtype=BF16, device="cuda")
    got = f64(D().linear(a, w, bias=torch.from_numpy(v).cuda(), act=act, out_dtype=F32))
    x = v.astype(np.float64)
    ref = OD.activate(x, act)
    off = np.abs(got - ref) - OD.activation_error(x, act) * OD.U * np.abs(ref) - 2.0 ** -145
    assert np.all(off <= 0), (act, v[off.max(0).argmax()])


# ---- block scales' first and last codes --------------------------------------------------

@pytest.mark.parametrize("M", [5, 40, 300])
@pytest.mark.parametrize("cw", [134, 247])
def test_block_scale_codes_0_and_255(M, cw):
    """Code 0 is 2^-127 and 255 is NaN, in the exact and in the scaled products, for
    blocks with elements (multiples of 2^-133 here) and for blocks of zeros."""
    rng = np.random.default_rng(M)
    N, K = 70, 256
    ca, cw_ = row_codes(M, K, rng), row_codes(N, K, rng)
    ca[1::3, 32:64] = 0                                        # blocks of zeros under code 0
    sa = np.where(rng.random((M, K // 32)) < 0.5, 254 - cw, 0).astype(np.uint8)
    sa[:, 1] = 0
    sa[0] = 0
    sw = np.full((N, K // 32), cw, np.uint8)
    sw[3, 5] = 0
    a_nan, w_nan = sa.copy(), sw.copy()
    a_nan[2, 7], w_nan[9, 0] = 255, 255
    for out in (F32, BF16):
        ops = lambda s, t: (D().FP8Rows(torch.from_numpy(ca).cuda(), torch.from_numpy(s).cuda()),
                            D().FP8Rows(torch.from_numpy(cw_).cuda(), torch.from_numpy(t).cuda()))
        ref, err = OD.linear(OD.dequantize(ca, sa), OD.dequantize(cw_, sw), scaled=out != F32)
        assert np.abs(ref[0]).max() > 0                        # a row of code 0 alone has values
        got = f64(D().linear(*ops(sa, sw), out_dtype=out))
        OD.check_rounded(got, ref, err + 2.0 ** -149, out)
        bad = f64(D().linear(*ops(a_nan, w_nan), out_dtype=out))
        want = np.zeros((M, N), bool)
        want[2], want[:, 9] = True, True
        assert np.array_equal(np.isnan(bad), want) and np.array_equal(bad[~want], got[~want])


# ---- launches in parts, threads, other allocators ----------------------------------------

def test_rows_past_one_launch():
    """2^21 rows fill one launch of the row operators: the next launch's first and last
    rows are as exact as the first one's."""
    T, K = 2 ** 21 + 37, 32
    x = torch.randn(T, K, generator=torch.Generator().manual_seed(1)).to(BF16)
    at = np.r_[0:40, 2 ** 21 - 40:T]
    xs = x[at].float().numpy()
    dx = x.cuda()
    for scales, oracle in (("row", OD.quantize_row), ("mx", OD.quantize_block)):
        q = D().quantize_fp8(dx, scales)
        c, s = oracle(xs)
        assert np.array_equal(q.codes.cpu().numpy()[at], c) and np.array_equal(q.scales.cpu().numpy()[at], s)
        r = D().rms_norm(dx, residual=dx, scales=scales)
        total = (2 * x.float()).to(BF16)
        assert torch.equal(r.total.cpu(), total)
        y, err = OD.rms_norm(f64(total[at]), None, 1e-6, 0.0)
        OD.check_rounded(f64(r.y)[at], y, err, BF16, scales)
        OD.check_fp8(r.fp8.codes.cpu().numpy()[at], r.fp8.scales.cpu().numpy()[at], y, err, scales)


def layer_calls(seed):
    g = torch.Generator().manual_seed(seed)
    x, h = (torch.randn(40, 256, generator=g).to(BF16).cuda() for _ in range(2))
    w = torch.randn(320, 256, generator=g).to(BF16).cuda()
    d = torch.randn(256, 160, generator=g).to(BF16).cuda()
    r = torch.randn(24, 256, generator=g).to(BF16).cuda()

    def run(mod):
        n = mod.rms_norm(x, residual=h, scales="mx")
        a = mod.linear(n.fp8, mod.quantize_fp8(w), act="gelu_tanh", gated=True, out_dtype="mx")
        out = mod.linear(a, mod.quantize_fp8(d), residual=n.total)
        return [n.y, n.total, *n.fp8, mod.linear(n.y, r, out_dtype=F32), *a, out, mod.quantize_fp8(x, "row").codes]
    return run


def test_threads_calling_at_once():
    """Threads with a stream each, calling at the same time, each get the results of
    their own inputs."""
    import threading
    D()
    calls = [layer_calls(s) for s in range(4)]
    want = [run(D()) for run in calls]
    torch.cuda.synchronize()
    got, go = [None] * 4, threading.Barrier(4)

    def work(i):
        try:
            stream = torch.cuda.Stream()
            with torch.cuda.stream(stream):
                go.wait(30)
                res = [calls[i](D()) for _ in range(15)]
            stream.synchronize()
            got[i] = res
        except Exception as e:
            got[i] = e
    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join(60)
    for g, w in zip(got, want):
        assert isinstance(g, list), g
        for res in g:
            assert all(torch.equal(p, q) for p, q in zip(res, w))


def test_without_torchs_own_shortcuts(monkeypatch):
    """Where torch lacks the private functions that small calls go through, the public
    ones give the same, on another stream as well."""
    import importlib.util
    assert D()._raw_stream is torch._C._cuda_getCurrentRawStream         # the shortcuts are taken here
    monkeypatch.delattr(torch._C, "_cuda_getCurrentRawStream")
    monkeypatch.delattr(torch._C, "_cuda_getDevice")
    monkeypatch.delattr(torch._C._dynamo.guards, "_empty_strided_cuda")
    spec = importlib.util.spec_from_file_location("nvfp4_w4a4_expert_amd.dense_public", D().__file__)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    monkeypatch.undo()
    assert mod._raw_stream is not D()._raw_stream and mod._empty_strided is not D()._empty_strided
    assert mod._raw_stream(0) == torch.cuda.current_stream().cuda_stream and mod._current_device() == 0
    run = layer_calls(9)
    want = run(D())
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(run(mod), want))
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        assert mod._raw_stream(0) == stream.cuda_stream
        got = run(mod)
    stream.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(got, want))


# ---- rows whose squares leave fp32's range -----------------------------------------------

@pytest.mark.parametrize("K", [24, 128, 256, 512, 1024, 2048, 4096, 8192, 16384, 32768])
def test_norm_of_rows_past_the_range_of_squares(K):
    """Finite rows of any size have the formula's values, side by side with ordinary
    rows, infinities and NaN (rows of one wavefront among them)."""
    rng = np.random.default_rng(K)
    sizes = [1.0, 1e30, 2.0 ** -66, 1e-30, 2.5e18, 3e19, 2.0 ** -110, 1.0, 1e25, 2.0 ** -128, 5e37, 1e-19, 1.0]
    x = torch.from_numpy(np.clip(rng.standard_normal((len(sizes), K)), -3, 3) * np.array(sizes)[:, None]).to(BF16)
    extra = torch.zeros(6, K, dtype=BF16)
    extra[0] = torch.finfo(BF16).max
    extra[1, 5], extra[1, 7] = 1e30, 1.0                       # one huge element
    extra[2] = 2.0 ** -133                                     # the smallest bf16 number
    extra[3, 9] = float("inf")
    extra[3, 2] = 1e30
    extra[4] = 1e30
    extra[4, 11] = float("nan")
    extra[5, 3] = -2.0 ** -133
    x = torch.cat([x, extra])
    bad = np.array([len(sizes) + 3, len(sizes) + 4])
    good = np.setdiff1d(np.arange(x.shape[0]), bad)
    w = torch.from_numpy(rng.standard_normal(K)).to(BF16)
    for eps in (0.0, 2.0 ** -90, 1e-6, 1e38):
        for scales in ("row", "mx") if K % 32 == 0 else ("row",):
            n = D().rms_norm(x.cuda(), w.cuda(), eps=eps, weight_offset=1.0, scales=scales)
            y, err = OD.rms_norm(f64(x)[good], f64(w), float(np.float32(eps)), 1.0)
            err = err + 2.0 ** -140
            OD.check_rounded(f64(n.y)[good], y, err, BF16, f"{K} {eps}")
            c, s = n.fp8.codes.cpu().numpy(), n.fp8.scales.cpu().numpy()
            # Row form: code = E4M3(y * min(1 / scale, FLT_MAX)).  Where scale = amax / 448 is below
            # 1 / FLT_MAX the second factor is less than 1 / scale, so code * scale lies between 0
            # and y up to the code's own rounding: off by up to |y| by definition.
            low = np.abs(y).max(1, keepdims=True) < 448 * 2.0 ** -128 * (1 + 2.0 ** -10)
            lost = np.where(low, np.abs(y), 0) if scales == "row" else 0
            OD.check_fp8(c[good], s[good], y, err, f"{K} {eps} {scales}", lost)
            z = f64(n.y)[bad]
            assert np.isnan(z[1]).all() and np.isnan(z[0, 9]) and not np.delete(z[0], 9).any()
            assert np.all((c[bad[1]] & 0x7F) == 0x7F) and not (np.delete(c[bad[0]], 9) & 0x7F).any()
