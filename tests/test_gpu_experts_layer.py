"""GPU tests of ExpertsLayer at the ends of its range: no tokens, one expert, all experts,
rows of other types than the layer's."""
import pytest
import torch

pytestmark = pytest.mark.gpu

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32


def X():
    from nvfp4_w4a4_expert_amd import experts
    return experts


def rand(shape, seed, dtype=BF16, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale).to(dtype).cuda()


def layer(kind, E=4, inter=32, H=64):
    w13, w2 = rand((E, 2 * inter, H), 1, BF16, H ** -0.5), rand((E, H, inter), 2, BF16, inter ** -0.5)
    return X().ExpertsLayer(w13, w2) if kind == "bf16" else X().ExpertsLayer.quantized(w13, w2, kind)


@pytest.mark.parametrize("kind", ["bf16", "row", "mx"])
def test_no_tokens(kind):
    out = layer(kind).forward(rand((0, 64), 3), rand((0, 4), 4, F32), 2, residual=rand((0, 64), 5))
    assert out.shape == (0, 64) and out.dtype == BF16


@pytest.mark.parametrize("kind", ["bf16", "row", "mx"])
@pytest.mark.parametrize("E,k", [(1, 1), (4, 4)])
def test_one_and_all_experts(kind, E, k):
    m, x, logits = layer(kind, E), rand((9, 64), 3), rand((9, E), 4, F32)
    out = m.forward(x, logits, k, out_dtype=F32)
    value = lambda q: q.float() if kind == "bf16" else q.dequantize()
    w13, w2 = value(m.w13), value(m.w2)
    p = torch.softmax(logits, 1)
    ref = torch.zeros(9, 64, device="cuda")
    for e in range(E):
        gate, up = (x.float() @ w13[e].t().contiguous()).chunk(2, 1)
        ref += p[:, e:e + 1] * ((torch.nn.functional.silu(gate) * up) @ w2[e].t().contiguous())
    # bf16: h's rounding, 2^-8 of each element.  8 bits: x's and h's, at most 2^-4 of each
    # element, uniform, so 2^-4 / sqrt(3) of the norm; x's acts through the gate (slope at
    # most 1.1) and up: sqrt(1.1^2 + 1 + 1) * 2^-4 / sqrt(3) = 0.065
    tol = 0.02 if kind == "bf16" else 0.1
    assert (out - ref).norm() <= tol * ref.norm()


def test_tokens_and_logits_that_do_not_belong_together():
    m, x = layer("bf16"), rand((9, 64), 3)
    for shape in ((10, 4), (8, 4), (9, 5)):
        with pytest.raises(ValueError, match="logits"):
            m.forward(x, rand(shape, 4, F32), 2)
    assert m.forward(x, rand((9, 4), 4, F32), 2).isfinite().all()
