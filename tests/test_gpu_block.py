"""GPU tests of block_norm against the float64 oracle: widths, gates, outputs, values
that are not finite or whose squares leave fp32's range, strides and guards, outputs
over inputs, offsets past 32 bits, streams and graph replays."""
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


def gate_of(kind, T, K, dtype, seed):
    shape = {"row": (T, 1), "channel": (K,), "channel2": (1, K), "full": (T, K), "one": (1,)}.get(kind)
    return None if kind == "none" else 0.375 if kind == "scalar" else rand(shape, seed, dtype, 1.5)


def check(n, x, r, want_y, scales, label, post=True, w_post=None, w=None, gate=None, act=None, rs=1.0, eps=1e-6, offset=0.0):
    """n against the oracle, the second norm over the total that came back."""
    dtype = x.dtype
    g = 1.0 if gate is None else f64(gate) if isinstance(gate, torch.Tensor) else gate
    t, err = OD.block_total(f64(x), f64(r), post, None if w_post is None else f64(w_post), eps, offset, g, act, rs)
    OD.check_rounded(f64(n.total), t, err, dtype, label + " total")
    y, err = OD.rms_norm(f64(n.total), None if w is None else f64(w), eps, offset)
    if want_y:
        OD.check_rounded(f64(n.y), y, err, dtype, label + " y")
    else:
        assert n.y is None
    if scales:
        OD.check_fp8(n.fp8.codes.cpu().numpy(), n.fp8.scales.cpu().numpy(), y, err, label)
    else:
        assert n.fp8 is None


def case(T, K, dtype, post=True, weights=True, gate="none", gate_dtype=None, act=None, rs=1.0, offset=0.0, scales=None, want_y=True,
         seed=0, eps=1e-6):
    x, r = rand((T, K), seed, dtype), rand((T, K), seed + 1, dtype, 3.0)
    x[:, :: max(1, K // 5)] *= 20
    w_post = rand((K,), seed + 2, dtype, 0.3) if weights and post else None
    w = rand((K,), seed + 3, dtype, 0.3) if weights and (want_y or scales) else None
    g = gate_of(gate, T, K, gate_dtype or dtype, seed + 4)
    up = lambda t: t.cuda() if isinstance(t, torch.Tensor) else t
    n = D().block_norm(up(x), up(r), post_norm=post, post_weight=up(w_post), gate=up(g), gate_act=act, residual_scale=rs, weight=up(w),
                       eps=eps, weight_offset=offset, want_y=want_y, scales=scales)
    check(n, x, r, want_y, scales, f"{T}x{K} {dtype} {gate} {act} {scales}", post, w_post, w, g, act, rs, eps, offset)


WIDTHS = [8, 24, 128, 136, 256, 264, 504, 512, 520, 1024, 1032, 2048, 2056, 2816, 4096, 4104, 8192, 8200, 16384, 16392, 32768]


@pytest.mark.parametrize("K", WIDTHS)
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_widths(K, dtype):
    for T, scales, gate in ((1, "row", "full"), (5, None, "channel"), (18, "row", "row")):
        case(T, K, dtype, gate=gate, rs=0.75, offset=1.0, scales=scales, seed=K + T)
    if K % 32 == 0:
        case(7, K, dtype, gate="scalar", rs=0.75, scales="mx", seed=K)


@pytest.mark.parametrize("gate,act", [(g, a) for g in ("none", "scalar", "one", "row", "channel", "channel2", "full")
                                      for a in (None, "sigmoid", "tanh") if a is None or g not in ("none", "scalar")])
@pytest.mark.parametrize("gate_dtype", [None, F32])
def test_gates(gate, act, gate_dtype):
    case(9, 704, BF16, gate=gate, gate_dtype=gate_dtype, act=act, rs=0.5, offset=1.0, scales="mx", seed=11)
    case(67, 136, F16, gate=gate, gate_dtype=gate_dtype, act=act, post=False, rs=-1.25, scales="row", seed=12)


@pytest.mark.parametrize("post,weights,scales,want_y", itertools.product([False, True], [False, True], [None, "row", "mx"], [False, True]))
def test_outputs(post, weights, scales, want_y):
    case(9, 704, BF16, post, weights, "channel", rs=0.8125, offset=0.5, scales=scales, want_y=want_y, seed=3)
    case(3, 2816, F16, post, weights, "row", act="sigmoid", scales=scales, want_y=want_y, seed=4)


def test_gates_at_the_ends_of_their_range():
    T, K = 12, 256
    x, r = rand((T, K), 1, BF16), torch.zeros(T, K, dtype=BF16)
    for dtype in (BF16, F32):
        g = torch.tensor([-200.0, -88.0, -60.0, -17.0, -1e-3, -0.0, 1e-30, 3e-3, 0.4, 9.0, 60.0, 3e38]).to(dtype)[:, None]
        for act in ("sigmoid", "tanh"):
            n = D().block_norm(x.cuda(), r.cuda(), gate=g.cuda(), gate_act=act, scales="row")
            check(n, x, r, True, "row", f"{act} {dtype}", gate=g, act=act)


def test_zero_rows_and_eps():
    x, r = torch.zeros(6, 96, dtype=BF16), torch.zeros(6, 96, dtype=BF16)
    x[1], r[2], x[3, 5] = 1.0, 2.0, 2.0 ** -60
    for eps in (1e-6, 2.5):
        for scales in ("row", "mx"):
            n = D().block_norm(x.cuda(), r.cuda(), eps=eps, scales=scales, residual_scale=0.5)
            check(n, x, r, True, scales, f"eps {eps}", rs=0.5, eps=eps)
            assert not n.total[0].any() and not n.y[0].any() and not n.fp8.codes[0].any()
    # a residual that the gate removes leaves the stream's own rows
    n = D().block_norm(x.cuda(), r.cuda(), gate=0.0)
    assert torch.equal(n.total.cpu(), r)


def test_values_that_are_not_finite_stay_in_their_rows():
    x, r = rand((6, 256), 1), rand((6, 256), 2)
    x[1, 7], x[3, 9], r[4, 11] = float("nan"), float("inf"), float("-inf")
    good = [0, 2, 5]
    for scales in ("row", "mx"):
        n = D().block_norm(x.cuda(), r.cuda(), scales=scales)
        t, y = n.total.cpu(), n.y.cpu().float()
        assert t[1].isnan().all() and y[1].isnan().all()
        # an infinity: NaN there, 0 elsewhere behind the first norm, so the residual stays
        rest = torch.arange(256) != 9
        assert t[3, 9].isnan() and torch.equal(t[3, rest], r[3, rest]) and y[3].isnan().all()
        # an infinite element of the total: NaN there, 0 elsewhere
        assert t[4, 11] == float("-inf") and y[4, 11].isnan() and not y[4, torch.arange(256) != 11].any()
        part = D().NormOut(n.y[good], n.total[good], D().FP8Rows(n.fp8.codes[good], n.fp8.scales[good]))
        check(part, x[good], r[good], True, scales, "finite rows")


@pytest.mark.parametrize("K", [64, 704, 2816, 8192])
def test_rows_whose_squares_leave_the_range(K):
    x, r = rand((4, K), 5), rand((4, K), 6)
    x[0], x[1], r[2], x[2] = x[0] * 2.0 ** 100, x[1] * 2.0 ** -80, r[2] * 2.0 ** 90, x[2] * 2.0 ** 90
    r[1] = 0
    n = D().block_norm(x.cuda(), r.cuda(), scales="row", eps=2.0 ** -140)
    check(n, x, r, True, "row", "wide range", eps=2.0 ** -140)
    n = D().block_norm(x.cuda(), r.cuda(), post_norm=False, scales="mx", eps=2.0 ** -140)
    check(n, x, r, True, "mx", "wide range, no first norm", post=False, eps=2.0 ** -140)


def test_strides_guards_and_outputs_over_inputs():
    T, K, pad = 37, 712, 24
    for dtype in (BF16, F16):
        big = [rand((T + 2, K + pad), s, dtype).cuda() for s in range(5)]
        x, r, out, tot, g = (b[1:T + 1, 8:8 + K] for b in big)
        keep = [b.clone() for b in big]
        w = rand((K,), 9, dtype, 0.3).cuda()
        n = D().block_norm(x, r, gate=g, weight=w, out=out, total_out=tot, scales="row", residual_scale=0.5)
        assert n.y is out and n.total is tot
        check(n, x, r, True, "row", "strides", w=w, gate=g, rs=0.5)
        for b, k in zip(big, keep):
            b[1:T + 1, 8:8 + K] = k[1:T + 1, 8:8 + K]
            assert torch.equal(b, k)
        ref = n.y.clone(), n.total.clone()
        # the same with the total over the residual, y over x, and the other way round
        ref = D().block_norm(x, r, gate=g, weight=w, residual_scale=0.5)
        for a, b in ((x, r), (r, x)):
            xs, rs = x.clone(), r.clone()
            x2, r2 = torch.empty_like(big[0]), torch.empty_like(big[0])
            xv, rv = x2[1:T + 1, 8:8 + K], r2[1:T + 1, 8:8 + K]
            xv.copy_(xs)
            rv.copy_(rs)
            n = D().block_norm(xv, rv, gate=g, weight=w, residual_scale=0.5, out=xv if a is x else rv, total_out=rv if a is x else xv)
            assert torch.equal(n.y, ref.y) and torch.equal(n.total, ref.total)


def test_empty_single_and_many_rows():
    e = torch.empty(0, 64, dtype=BF16, device="cuda")
    n = D().block_norm(e, e, gate=torch.empty(0, 1, dtype=BF16, device="cuda"), scales="mx")
    assert n.y.shape == (0, 64) and n.total.shape == (0, 64) and n.fp8.scales.shape == (0, 2)
    case(1, 2816, BF16, gate="full", scales="mx")
    T = (1 << 21) + 1003                                       # more than one launch holds
    x = rand((T, 8), 1).cuda()
    n = D().block_norm(x, x, gate=0.5, want_y=False)
    one = D().block_norm(x[-1003:].contiguous(), x[-1003:].contiguous(), gate=0.5, want_y=False)
    assert torch.equal(n.total[-1003:], one.total)
    assert torch.equal(n.total[:1003], D().block_norm(x[:1003], x[:1003], gate=0.5, want_y=False).total)


def test_offsets_past_32_bits():
    T, K = 70, 32
    ld = (1 << 31) // 64 + 8                                   # row 64 starts past 2^31 elements
    buf = torch.zeros((T - 1) * ld + K, dtype=BF16, device="cuda")
    x = torch.as_strided(buf, (T, K), (ld, 1))
    x.copy_(rand((T, K), 3))
    r = rand((T, K), 4).cuda()
    n = D().block_norm(x, r, total_out=x)
    check(n, rand((T, K), 3), r.cpu(), True, None, "far rows")


def test_streams_and_graph_replays():
    T, K = 33, 2816
    x, r, w = rand((T, K), 1).cuda(), rand((T, K), 2).cuda(), rand((K,), 3, BF16, 0.3).cuda()
    g = rand((T, 1), 4).cuda()
    call = lambda s=None: D().block_norm(x, r, post_weight=w, gate=g, gate_act="sigmoid", weight=w, scales="mx", stream=s)
    ref = call()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = call(side)
    raw = call(side.cuda_stream)
    side.synchronize()
    for n in (got, raw):
        assert torch.equal(n.y, ref.y) and torch.equal(n.total, ref.total) and torch.equal(n.fp8.codes, ref.fp8.codes)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        n = call()
    for seed in range(3):
        x.copy_(rand((T, K), 10 + seed))
        graph.replay()
        torch.cuda.synchronize()
        ref = call()
        assert torch.equal(n.y, ref.y) and torch.equal(n.total, ref.total) and torch.equal(n.fp8.codes, ref.fp8.codes) and \
            torch.equal(n.fp8.scales, ref.fp8.scales)


def test_plain_gate_is_the_norm_with_residual():
    """Without a first norm, gate and scale, the total is rms_norm's to the bit."""
    x, r, w = rand((29, 704), 1).cuda(), rand((29, 704), 2).cuda(), rand((704,), 3).cuda()
    a = D().block_norm(x, r, post_norm=False, weight=w, weight_offset=1.0, scales="row")
    b = D().rms_norm(x, w, residual=r, weight_offset=1.0, scales="row")
    assert torch.equal(a.total, b.total) and torch.equal(a.y, b.y) and torch.equal(a.fp8.codes, b.fp8.codes)
