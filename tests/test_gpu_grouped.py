"""GPU tests of experts.grouped_linear and ExpertsLayer against the float64 oracle:
types, group sizes from none to many tiles, gathered rows, outputs, strides and guards,
offsets past 32 bits, malformed offsets and indexes, streams, replays, the whole layer."""
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


def X():
    from nvfp4_w4a4_expert_amd import experts
    return experts


def rand(shape, seed, dtype=BF16, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale).to(dtype)


def f64(t):
    return t.detach().cpu().double().numpy()


def operand(shape, seed, kind, scale):
    """(operand on the GPU, its float64 values) of [rows, K] or [experts, rows, K]."""
    flat = (-1, shape[-1])
    if kind in ("bf16", "fp16"):
        t = rand(shape, seed, BF16 if kind == "bf16" else F16, scale)
        return t.cuda(), f64(t)
    q = D().quantize_fp8(rand(shape, seed, BF16, scale).reshape(flat).contiguous().cuda(), kind)
    v = OD.dequantize(q.codes.cpu().numpy(), q.scales.cpu().numpy()).reshape(shape)
    return D().FP8Rows(*(t.view(*shape[:-1], *t.shape[1:]) for t in q)), v


def is_scaled(kind, out):
    return kind in ("row", "mx") and out in (None, BF16, F16)


def offsets_of(sizes, first=0):
    return torch.tensor([first] + list(first + np.cumsum(sizes)), dtype=torch.int32)


def check_groups(got, av, wv, sizes, rows, kind, out, bias=None, act=None, gated=False, first=0, label=""):
    at = first
    for e, n in enumerate(sizes):
        if n == 0:
            continue
        ref, err = OD.linear(av[rows[at:at + n]], wv[e], None if bias is None else f64(bias[e]), act, gated, None,
                             is_scaled(kind, out))
        name = f"{label} expert {e} of {n} rows"
        if out == "mx":
            OD.check_fp8(got.codes[at:at + n].cpu().numpy(), got.scales[at:at + n].cpu().numpy(), ref, err, name)
        else:
            OD.check_rounded(f64(got[at:at + n]), ref, err, got.dtype, name)
        at += n


def case(sizes, N, K, kind, act=None, gated=False, bias=None, out=None, top=None, seed=0):
    E, P = len(sizes), int(sum(sizes))
    T = P if top is None else max(1, -(-P // top))
    a, av = operand((T, K), seed, kind, 1.0)
    w, wv = operand((E, 2 * N if gated else N, K), seed + 1, kind, K ** -0.5)
    b = None if bias is None else rand((E, 2 * N if gated else N), seed + 2, bias, 0.5)
    rows, index = np.arange(P), None
    if top is not None:
        pairs = torch.randperm(T * top, generator=torch.Generator().manual_seed(seed + 3))[:P].int()
        rows, index = (pairs // top).numpy(), pairs.cuda()
    got = X().grouped_linear(a, w, offsets_of(sizes).cuda(), index=index, index_div=top or 1, bias=None if b is None else b.cuda(),
                             act=act, gated=gated, out_dtype=out)
    if out != "mx":
        assert got.shape == (P, N) and got.dtype == (out or (F16 if kind == "fp16" else BF16))
    check_groups(got, av, wv, sizes, rows, kind, out, b, act, gated, label=f"{N}x{K} {kind} {act} gated={gated} {out} top={top}")


KINDS = ["bf16", "fp16", "row", "mx"]
# means of the rows from one to many; groups without a row, of one, that fill tiles, that
# pass them by one
SIZES = {
    "few": [[1], [16], [1, 0, 1, 3], [0, 0, 5], [17, 0, 1, 2, 33, 0, 0, 0], [2] * 70],
    "middle": [[17], [64], [65], [0, 100, 0, 64, 1, 0, 63, 65], [96, 0], [1, 300, 0, 1, 2]],
    "large": [[97], [128, 0, 256], [129, 1, 511, 0, 127], [1000], [0, 0, 0, 777, 0]],
}


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("which", list(SIZES))
@pytest.mark.parametrize("top", [None, 3])
def test_group_sizes(kind, which, top):
    for i, sizes in enumerate(SIZES[which]):
        for N, K in (((1, 32), (33, 96), (130, 416))[i % 3], (64, 128)):
            case(sizes, N, K, kind, top=top, seed=i)


@pytest.mark.parametrize("kind,K", [("bf16", 8), ("bf16", 72), ("fp16", 200), ("row", 16), ("row", 144), ("mx", 32), ("mx", 160), ("mx", 544),
                                    ("bf16", 2816), ("mx", 2112)])
def test_depths(kind, K):
    for sizes in ([3, 0, 9], [40, 30, 0, 20], [260, 0, 140]):
        case(sizes, 33, K, kind, seed=K)
        case(sizes, 70, K, kind, gated=True, act="silu", out=F32, top=2, seed=K + 1)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("out", [BF16, F16, F32, "mx"])
@pytest.mark.parametrize("gated", [False, True])
def test_outputs(kind, out, gated):
    acts = itertools.cycle([None, "silu", "gelu", "gelu_tanh", "relu"])
    for i, (sizes, N) in enumerate((([4, 0, 7], 96), ([50, 33, 0], 224), ([300, 0, 200], 160))):
        case(sizes, N, 224, kind, next(acts), gated, [None, F32, BF16][i], out, top=[None, 2, 4][i], seed=i)
        case(sizes, N, 224, kind, next(acts), gated, [F16, None, F32][i], out, seed=i)


@pytest.mark.parametrize("kind,N,K,gated", [("bf16", 3200, 96, False), ("fp16", 1700, 64, True), ("row", 3333, 144, False), ("mx", 1600, 160, True),
                                            ("mx", 3200, 608, False)])
def test_wide_results(kind, N, K, gated):
    """Enough columns for the larger tiles at every number of rows: partly empty tiles,
    columns that end in a tile's first half, more and less than the steps on their way."""
    g = torch.Generator().manual_seed(N)
    for E, most in ((23, 2), (25, 40), (21, 140), (17, 300), (11, 700)):
        sizes = (torch.randint(0, most + 1, (E,), generator=g)).tolist()
        case(sizes, N, K, kind, gated=gated, act="silu" if gated else None, top=3 if E % 4 == 1 else None, seed=E)
        if E == 25:
            case(sizes, N // 32 * 32, K, kind, gated=gated, out="mx", seed=E)
            case(sizes, N, K, kind, gated=gated, bias=F32, out=F32, seed=E)


def test_many_experts():
    g = torch.Generator().manual_seed(5)
    for E in (63, 64, 65, 128, 1000, 1024):
        sizes = (torch.randint(0, 3, (E,), generator=g) * torch.randint(0, 2, (E,), generator=g)).tolist()
        case(sizes, 16, 64, "bf16", seed=E)
    sizes = [0] * 1024
    sizes[1023], sizes[0], sizes[500] = 40000, 1, 3
    case(sizes, 16, 32, "bf16", seed=7)
    case(torch.randint(0, 60, (130,), generator=g).tolist(), 40, 64, "fp16", seed=8)


@pytest.mark.parametrize("kind", ["bf16", "mx"])
@pytest.mark.parametrize("sizes", [[3, 0, 4], [40, 0, 41], [150, 0, 151]])
def test_rows_outside_the_groups_stay(kind, sizes):
    first, behind, N, K = 5, 9, 40, 96
    P = first + sum(sizes) + behind
    a, av = operand((P, K), 1, kind, 1.0)
    w, wv = operand((len(sizes), N, K), 2, kind, 0.1)
    buf = torch.full((P + 2, N + 6), 7.0, dtype=BF16, device="cuda")
    out = buf[1:P + 1, 3:3 + N]
    X().grouped_linear(a, w, offsets_of(sizes, first).cuda(), out=out)
    check_groups(out, av, wv, sizes, np.arange(P), kind, BF16, first=first, label="outside")
    out[first:first + sum(sizes)] = 7.0
    assert (buf == 7.0).all()


@pytest.mark.parametrize("sizes", [[3, 0, 4], [40, 0, 41], [150, 0, 151]])
def test_indexes_outside_a_leave_their_rows(sizes):
    P, T, N, K = sum(sizes), 11, 40, 96
    for kind in ("bf16", "row", "mx"):
        a, av = operand((T, K), 1, kind, 1.0)
        w, wv = operand((len(sizes), N, K), 2, kind, 0.1)
        index = torch.randint(0, 2 * T, (P,), generator=torch.Generator().manual_seed(1)).int()
        bad = torch.zeros(P, dtype=torch.bool)
        for i, v in ((0, -1), (2, 2 * T), (P - 1, 2 ** 31 - 1), (4, -2 ** 31)):
            index[i], bad[i] = v, True
        out = torch.full((P, N), 7.0, dtype=F32, device="cuda")
        X().grouped_linear(a, w, offsets_of(sizes).cuda(), index=index.cuda(), index_div=2, out=out)
        assert (out[bad.cuda()] == 7.0).all()
        good = out.clone()
        ref = X().grouped_linear(a, w, offsets_of(sizes).cuda(), index=torch.where(bad, 0, index).int().cuda(), index_div=2, out_dtype=F32)
        good[bad.cuda()] = ref[bad.cuda()]
        assert torch.equal(good, ref)
        check_groups(ref, av, wv, sizes, (torch.where(bad, 0, index) // 2).numpy(), kind, F32, label="indexes")
        empty = a[:0] if isinstance(a, torch.Tensor) else D().FP8Rows(a.codes[:0], a.scales[:0])
        keep = torch.full((P, N), 7.0, device="cuda")
        X().grouped_linear(empty, w, offsets_of(sizes).cuda(), index=index.cuda(), out=keep)
        assert (keep == 7.0).all()


@pytest.mark.parametrize("offsets", [[0, 50, 20, 90], [-5, 30, 60, 200], [90, 60, 30, 0], [2 ** 31 - 1, -2 ** 31, 5, 90], [40, 40, 40, 40]])
def test_malformed_offsets_stay_inside(offsets):
    P, N, K = 90, 40, 64
    a, w = rand((P, K), 1).cuda(), rand((3, N, K), 2).cuda()
    for rows in (P, 40):                                       # (64-row tiles, few rows)
        buf = torch.full((rows + 40, N), 7.0, dtype=BF16, device="cuda")
        X().grouped_linear(a[:rows], w, torch.tensor(offsets, dtype=torch.int32).cuda(), out=buf[20:20 + rows])
        assert (buf[:20] == 7.0).all() and (buf[20 + rows:] == 7.0).all()
        each = [a[:rows].float() @ w[e].float().t() for e in range(3)]
        got = buf[20:20 + rows].float()
        ok = (got == 7.0).all(1)
        for v in each:
            ok |= ((got - v).abs() < 0.05 + 0.01 * v.abs()).all(1)
        assert ok.all()


def test_strides_of_a_and_weights():
    sizes, N, K = [70, 0, 90], 48, 104
    for dtype in (BF16, F16):
        a = rand((160, K + 24), 1, dtype).cuda()[:, 8:8 + K]
        big = rand((6, N + 3, K + 16), 2, dtype, 0.1).cuda()
        w = big[::2, 1:1 + N, 8:8 + K]
        got = X().grouped_linear(a, w, offsets_of(sizes).cuda(), act="silu")
        assert torch.equal(got, X().grouped_linear(a.contiguous(), w.contiguous(), offsets_of(sizes).cuda(), act="silu"))
    one = w[1:2]
    got = X().grouped_linear(a, one, torch.tensor([0, 160], dtype=torch.int32).cuda())
    assert torch.equal(got, X().grouped_linear(a, one.contiguous(), torch.tensor([0, 160], dtype=torch.int32).cuda()))


@pytest.mark.parametrize("sizes", [[5, 0, 7], [30, 0, 40], [0, 210, 140]])
def test_offsets_past_32_bits(sizes):
    N, K, P = 24, 32, sum(sizes)
    far = (1 << 31) + 64                                       # elements between experts: 4 GiB
    wb = torch.zeros(2 * far + N * K, dtype=BF16, device="cuda")
    w = torch.as_strided(wb, (3, N, K), (far, K, 1))
    w.copy_(rand((3, N, K), 1, BF16, 0.2))
    ld = (1 << 22)                                             # 8 MiB rows of a and of the result
    T = 600
    ab = torch.zeros((T - 1) * ld + K, dtype=BF16, device="cuda")
    a = torch.as_strided(ab, (T, K), (ld, 1))
    a.copy_(rand((T, K), 2))
    index = torch.randint(0, T, (P,), generator=torch.Generator().manual_seed(3)).int()
    index[0] = T - 1
    ref = X().grouped_linear(a.contiguous(), w.contiguous(), offsets_of(sizes).cuda(), index=index.cuda(), out_dtype=F32)
    ob = torch.zeros((P - 1) * (1 << 24) // 2 + N, dtype=F32, device="cuda") if P < 100 else None
    out = None if ob is None else torch.as_strided(ob, (P, N), ((1 << 24) // 2, 1))
    got = X().grouped_linear(a, w, offsets_of(sizes).cuda(), index=index.cuda(), out_dtype=F32, out=out)
    assert torch.equal(got, ref)


def test_equal_to_linear_with_one_expert():
    for kind in KINDS:
        for M in (200, 150, 9):
            a, _ = operand((M, 352), 1, kind, 1.0)
            w, _ = operand((1, 96, 352), 2, kind, 0.05)
            w2 = w[0] if isinstance(w, torch.Tensor) else D().FP8Rows(w.codes[0], w.scales[0])
            got = X().grouped_linear(a, w, torch.tensor([0, M], dtype=torch.int32).cuda(), out_dtype=F32)
            assert torch.allclose(got, D().linear(a, w2, out_dtype=F32), rtol=0, atol=1e-5)


def test_values_that_are_not_finite_stay_in_their_rows():
    for sizes in ([3, 4], [40, 41], [130, 140]):
        P, K = sum(sizes), 96
        a, w = rand((P, K), 1), rand((2, 40, K), 2, BF16, 0.1)
        ref = X().grouped_linear(a.cuda(), w.cuda(), offsets_of(sizes).cuda())
        a[1, 5], a[P - 1, 0] = float("nan"), float("inf")
        got = X().grouped_linear(a.cuda(), w.cuda(), offsets_of(sizes).cuda())
        assert got[1].isnan().all() and not got[P - 1].isfinite().any()
        keep = [i for i in range(P) if i not in (1, P - 1)]
        assert torch.equal(got[keep], ref[keep])


def test_streams_replays_and_repeats():
    for sizes in ([3, 0, 9, 1], [60, 0, 70], [300, 200, 0]):
        P, N, K = sum(sizes), 64, 256
        a, w, o = rand((P, K), 1).cuda(), rand((len(sizes), 2 * N, K), 2, BF16, 0.1).cuda(), offsets_of(sizes).cuda()
        index = torch.randperm(P, generator=torch.Generator().manual_seed(1)).int().cuda()
        call = lambda s=None: X().grouped_linear(a, w, o, index=index, act="silu", gated=True, out_dtype="mx", stream=s)
        ref = call()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        got, raw = call(side), call(side.cuda_stream)
        side.synchronize()
        for q in (got, raw):
            assert torch.equal(q.codes, ref.codes) and torch.equal(q.scales, ref.scales)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = call()
        for s in range(3):
            a.copy_(rand((P, K), 10 + s))
            moved = list(np.roll(sizes, s))                    # the groups may change between replays
            o.copy_(offsets_of(moved))
            graph.replay()
            torch.cuda.synchronize()
            ref = call()
            assert torch.equal(got.codes, ref.codes) and torch.equal(got.scales, ref.scales)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("T", [1, 16, 700])
def test_experts_layer(kind, T):
    """route -> permute -> gate/up -> down -> combine, stage by stage and as a layer."""
    E, k, H, I = 16, 3, 256, 96
    dtype = F16 if kind == "fp16" else BF16
    x, r = rand((T, H), 1, dtype).cuda(), rand((T, H), 2, dtype).cuda()
    logits = rand((T, E), 3, F32).cuda()
    w13, w2 = rand((E, 2 * I, H), 4, dtype, H ** -0.5).cuda(), rand((E, H, I), 5, dtype, I ** -0.5).cuda()
    b13, b2 = rand((E, 2 * I), 6, F32, 0.3).cuda(), rand((E, H), 7, F32, 0.3).cuda()
    if kind in ("row", "mx"):
        layer = X().ExpertsLayer.quantized(w13, w2, kind, act="gelu_tanh", bias13=b13, bias2=b2)
    else:
        layer = X().ExpertsLayer(w13, w2, act="gelu_tanh", bias13=b13, bias2=b2)
    out = layer.forward(x, logits, k, residual=r)
    assert out.dtype == dtype and out.shape == (T, H)
    xq = x if layer.scales is None else D().quantize_fp8(x, kind)
    assert torch.equal(layer.forward(xq, logits, k, residual=r, out_dtype=dtype), out)
    rt = X().route(logits, k)
    g = X().permute(rt.ids, E)
    h = X().grouped_linear(xq, layer.w13, g.offsets, index=g.src_pair, index_div=k, bias=b13, act="gelu_tanh", gated=True,
                           out_dtype="mx" if kind == "mx" else None)
    hq = D().quantize_fp8(h, "row") if kind == "row" else h
    v = X().grouped_linear(hq, layer.w2, g.offsets, bias=b2, out_dtype=F32)
    assert torch.equal(X().combine(v, rt.weights, g.inv_pair, residual=r, out_dtype=dtype), out)
    val = lambda q: f64(q) if isinstance(q, torch.Tensor) else OD.dequantize(q.codes.cpu().numpy().reshape(-1, q.codes.shape[-1]),
                                                                             q.scales.cpu().numpy().reshape(-1, *q.scales.shape[q.codes.dim() - 1:])).reshape(q.codes.shape)
    o, src = g.offsets.cpu().numpy(), g.src_pair.cpu().numpy()
    sizes = np.diff(o).tolist()
    check_groups(h, val(xq), val(layer.w13), sizes, src // k, kind, "mx" if kind == "mx" else None, b13, "gelu_tanh", True, label="gate/up")
    check_groups(v, val(hq), val(layer.w2), sizes, np.arange(T * k), kind, F32, b2, label="down")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = layer.forward(x, logits, k, residual=r, stream=side)
    side.synchronize()
    assert torch.equal(other, out)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = layer.forward(x, logits, k, residual=r)
    for s in range(3):
        logits.copy_(rand((T, E), 20 + s, F32))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(got, layer.forward(x, logits, k, residual=r))
