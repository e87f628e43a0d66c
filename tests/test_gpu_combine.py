"""GPU tests of experts.route, permute and combine: the routing steps against torch's
sort, the combine against the float64 oracle."""
import itertools

import numpy as np
import pytest
import torch

from oracle import dense as OD

pytestmark = pytest.mark.gpu

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32


def X():
    from nvfp4_w4a4_expert_amd import experts
    return experts


def rand(shape, seed, dtype=BF16, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale).to(dtype)


def f64(t):
    return t.detach().cpu().double().numpy()


def check(got, v, w, inv, r, label):
    ref, err = OD.combine(f64(v), f64(w), inv.cpu().numpy(), None if r is None else f64(r))
    OD.check_rounded(f64(got), ref, err, got.dtype, label)


@pytest.mark.parametrize("dtype,out,res", itertools.product([BF16, F16, F32], [BF16, F16, F32], [None, BF16, F32]))
def test_combine_types(dtype, out, res):
    for T, k, H in ((1, 1, 8), (5, 3, 264), (33, 8, 704), (7, 9, 2816), (2, 33, 16)):
        v, w = rand((T * k, H), T, dtype), torch.softmax(rand((T, k), 2, F32), 1)
        inv = torch.randperm(T * k, generator=torch.Generator().manual_seed(k)).int()
        r = None if res is None else rand((T, H), 5, res)
        got = X().combine(v.cuda(), w.cuda(), inv.cuda(), residual=None if r is None else r.cuda(), out_dtype=out)
        check(got, v, w, inv, r, f"{T} {k} {H} {dtype} {out} {res}")


def test_left_out_pairs_and_repeated_rows():
    T, k, H = 21, 4, 40
    v, w = rand((30, H), 1), rand((T, k), 2, F32)
    inv = torch.randint(-3, 35, (T, k), generator=torch.Generator().manual_seed(3)).int()
    inv[4], inv[5, 2], inv[6, 1] = -1, 2 ** 31 - 1, -2 ** 31
    v[0] = float("inf")                                        # (what out-of-range pairs must not touch)
    inv[inv == 0] = 7
    r = rand((T, H), 4)
    got = X().combine(v.cuda(), w.cuda(), inv.cuda(), residual=r.cuda())
    check(got, v, w, inv, r, "left out")
    assert torch.equal(got[4].cpu(), r[4])
    none = X().combine(v[:0].cuda(), w.cuda(), inv.cuda(), residual=r.cuda())
    assert torch.equal(none.cpu(), r)
    assert X().combine(v.cuda(), w[:0].cuda(), inv[:0].cuda()).shape == (0, H)


def test_strides_out_and_residual_in_place():
    T, k, H = 19, 3, 72
    vb, rb = rand((T * k, H + 8), 1, F16).cuda(), rand((T + 2, H + 16), 2, F32).cuda()
    v, r = vb[:, 8:], rb[1:T + 1, 8:8 + H]
    w, inv = rand((T, k), 3, F32).cuda(), torch.arange(T * k).int().cuda()
    ref = X().combine(v, w, inv, residual=r, out_dtype=F32)
    keep = rb.clone()
    assert X().combine(v, w, inv, residual=r, out=r) is r
    assert torch.equal(r, ref)
    rb[1:T + 1, 8:8 + H] = keep[1:T + 1, 8:8 + H]
    assert torch.equal(rb, keep)


def test_values_past_32_bits():
    H, rows = 8, 40
    ld = (1 << 31) // 32 + 8
    buf = torch.zeros((rows - 1) * ld + H, dtype=BF16, device="cuda")
    v = torch.as_strided(buf, (rows, H), (ld, 1))
    v.copy_(rand((rows, H), 3))
    w, inv = rand((10, 4), 1, F32), torch.randperm(rows, generator=torch.Generator().manual_seed(1)).int()
    check(X().combine(v, w.cuda(), inv.cuda()), rand((rows, H), 3), w, inv, None, "far rows")


@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (5, 7, 3), (300, 128, 8), (64, 4, 4), (2000, 1024, 2)])
def test_route_and_permute(T, E, k):
    logits = rand((T, E), 1, F32)
    r = X().route(logits.cuda(), k)
    order = torch.sort(logits, dim=1, descending=True, stable=True).indices[:, :k]
    assert torch.equal(r.ids.cpu(), order.int())
    ref = torch.softmax(torch.gather(logits.double(), 1, order), 1)
    assert (r.weights.cpu().double() - ref).abs().max() < 1e-6
    ids = order.int().clone()
    ids[0, 0] = -1                                             # left out
    g = X().permute(ids.cuda(), E)
    flat = ids.reshape(-1)
    keep = torch.sort(torch.where(flat < 0, E, flat), stable=True).indices[:int((flat >= 0).sum())]
    n = keep.numel()
    assert torch.equal(g.src_pair[:n].cpu(), keep.int()) and (g.src_pair[n:] == -1).all()
    inv = torch.full((T * k,), -1, dtype=torch.int32)
    inv[keep] = torch.arange(n, dtype=torch.int32)
    assert torch.equal(g.inv_pair.cpu(), inv)
    counts = torch.bincount(flat[flat >= 0].long(), minlength=E)
    assert torch.equal(g.offsets.cpu(), torch.cat([torch.zeros(1, dtype=torch.long), counts.cumsum(0)]).int())


def test_combine_on_streams_and_replayed():
    T, k, H = 16, 8, 2816
    v, w = rand((T * k, H), 1, F32).cuda(), torch.softmax(rand((T, k), 2, F32), 1).cuda()
    inv = torch.randperm(T * k, generator=torch.Generator().manual_seed(1)).int().cuda()
    r = rand((T, H), 3).cuda()
    ref = X().combine(v, w, inv, residual=r)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = X().combine(v, w, inv, residual=r, stream=side)
    side.synchronize()
    assert torch.equal(got, ref)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = X().combine(v, w, inv, residual=r)
    for s in range(3):
        v.copy_(rand((T * k, H), 10 + s, F32))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(got, X().combine(v, w, inv, residual=r))
