"""GPU tests of block_norm's groups of threads with many rows, where launches take other
groups than with few, and of rows that are not finite or leave fp32's range in groups of
several wavefronts; against the float64 oracle."""
import pytest
import torch

from oracle import dense as OD

pytestmark = pytest.mark.gpu

BF16, F16 = torch.bfloat16, torch.float16


def D():
    from nvfp4_w4a4_expert_amd import dense
    return dense


def rand(shape, seed, dtype=BF16, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale).to(dtype)


def f64(t):
    return t.detach().cpu().double().numpy()


def check(n, x, r, w_post, w, scales, label, eps=1e-6):
    t, err = OD.block_total(f64(x), f64(r), True, f64(w_post), eps, 1.0, 1.0, None, 0.75)
    OD.check_rounded(f64(n.total), t, err, x.dtype, label + " total")
    y, err = OD.rms_norm(f64(n.total), f64(w), eps, 1.0)
    OD.check_rounded(f64(n.y), y, err, x.dtype, label + " y")
    if scales:
        OD.check_fp8(n.fp8.codes.cpu().numpy(), n.fp8.scales.cpu().numpy(), y, err, label)


def call(x, r, w_post, w, scales, eps=1e-6):
    return D().block_norm(x.cuda(), r.cuda(), post_weight=w_post.cuda(), weight=w.cuda(), weight_offset=1.0, residual_scale=0.75,
                          scales=scales, eps=eps)


# up to 512 rows and beyond them: 512 threads of a vector, 128 of three (the third full to
# empty), 256 of two; and the widths on either side
@pytest.mark.parametrize("K", [2048, 2056, 2080, 2816, 3064, 3080, 4096, 4104])
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_many_rows(K, dtype):
    w_post, w = rand((K,), 1, dtype, 0.3), rand((K,), 2, dtype, 0.3)
    x, r = rand((601, K), 3, dtype), rand((601, K), 4, dtype, 3.0)
    x[:, ::701] *= 20
    ref = None
    for scales in ("row", "mx", None) if K % 32 == 0 else ("row", None):
        n = call(x, r, w_post, w, scales)
        check(n, x, r, w_post, w, scales, f"{K} {dtype} {scales}")
        if ref is not None:
            assert torch.equal(n.total, ref.total) and torch.equal(n.y, ref.y)
        ref = n
    # both sides of the border give every row's values
    for rows in (512, 513):
        n = call(x[:rows], r[:rows], w_post, w, "row")
        check(n, x[:rows], r[:rows], w_post, w, "row", f"{rows} x {K}")


WIDE = [(6, 704), (6, 2816), (530, 2816), (6, 3080), (530, 3080), (6, 8192)]


@pytest.mark.parametrize("T,K", WIDE)
@pytest.mark.parametrize("scales", ["row", "mx"])
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_values_that_are_not_finite_stay_in_their_rows(T, K, scales, dtype):
    if scales == "mx" and K % 32:
        K += 24
    w_post, w = rand((K,), 1, dtype, 0.3), rand((K,), 2, dtype, 0.3)
    x, r = rand((T, K), 3, dtype), rand((T, K), 4, dtype, 3.0)
    nan, big, low = 1, T - 3, T - 2
    x[nan, K - 1], r[big, K // 2], r[low, 5] = float("nan"), float("inf"), float("-inf")
    n = call(x, r, w_post, w, scales)
    codes, y = n.fp8.codes.cpu(), n.y.cpu().float()
    assert y[nan].isnan().all() and ((codes[nan] & 0x7F) == 0x7F).all()
    # an infinite element of the total: NaN there, 0 elsewhere, and so its codes
    for row, at in ((big, K // 2), (low, 5)):
        rest = torch.arange(K) != at
        assert y[row, at].isnan() and not y[row, rest].any()
        assert (codes[row, at] & 0x7F) == 0x7F and not (codes[row, rest] & 0x7F).any()
    keep = torch.tensor([i for i in range(T) if i not in (nan, big, low)])
    on = keep.cuda()
    part = D().NormOut(n.y[on], n.total[on], D().FP8Rows(n.fp8.codes[on], n.fp8.scales[on]))
    check(part, x[keep], r[keep], w_post, w, scales, "finite rows")
    # and give what they give without the others
    x[[nan, big, low]], r[[nan, big, low]] = 0, 0
    ref = call(x, r, w_post, w, scales)
    assert torch.equal(ref.y[on], n.y[on]) and torch.equal(ref.fp8.codes[on], n.fp8.codes[on]) and torch.equal(ref.fp8.scales[on], n.fp8.scales[on])


@pytest.mark.parametrize("T,K", WIDE)
@pytest.mark.parametrize("scales", ["row", "mx"])
def test_rows_whose_squares_leave_the_range(T, K, scales):
    if scales == "mx" and K % 32:
        K += 24
    w_post, w = rand((K,), 1, BF16, 0.3), rand((K,), 2, BF16, 0.3)
    x, r = rand((T, K), 3), rand((T, K), 4, BF16, 3.0)
    x[0], x[T - 1], r[2], x[2] = x[0] * 2.0 ** 100, x[T - 1] * 2.0 ** -80, r[2] * 2.0 ** 90, x[2] * 2.0 ** 90
    r[T - 1] = 0
    check(call(x, r, w_post, w, scales, 2.0 ** -140), x, r, w_post, w, scales, f"{T} x {K}", 2.0 ** -140)
