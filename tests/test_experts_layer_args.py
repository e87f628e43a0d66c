"""Argument checks of ExpertsLayer, without a GPU."""
import pytest
import torch

from nvfp4_w4a4_expert_amd import dense as D
from nvfp4_w4a4_expert_amd import experts as X

BF16, F16, F32, U8 = torch.bfloat16, torch.float16, torch.float32, torch.uint8
T, E, I, H = 5, 3, 32, 64


def w(*shape, dtype=BF16):
    return torch.zeros(shape, dtype=dtype)


def f8(rows, K, row=True, experts=E):
    return D.FP8Rows(w(experts, rows, K, dtype=U8), w(experts, rows, dtype=F32) if row else w(experts, rows, K // 32, dtype=U8))


def layer(**kw):
    a = dict(w13=w(E, 2 * I, H), w2=w(E, H, I))
    a.update(kw)
    return X.ExpertsLayer(a.pop("w13"), a.pop("w2"), **a)


WELL = [{}, dict(w13=w(E, 2 * I, H, dtype=F16), w2=w(E, H, I, dtype=F16)), dict(w13=f8(2 * I, H), w2=f8(H, I)),
        dict(w13=f8(2 * I, H, False), w2=tuple(f8(H, I, False))), dict(bias13=w(E, 2 * I, dtype=F32), bias2=w(E, H), act=None),
        dict(w13=w(1, 2 * I, H).expand(1, 2 * I, H), w2=w(1, H, I)), dict(w13=w(2 * E, 2 * I, H + 8)[::2, :, :H], act="gelu")]


@pytest.mark.parametrize("kw", WELL)
def test_well_formed_layers_reach_the_device_check(kw):
    m = layer(**kw)
    assert m.num_experts == (kw["w13"].shape[0] if isinstance(kw.get("w13"), torch.Tensor) else E)
    x = w(T, H, dtype=m.w13.dtype if m.scales is None else BF16)
    with pytest.raises(ValueError, match="on a GPU"):
        m.forward(x, w(T, m.num_experts, dtype=F32), 1)
    if m.scales:
        one = f8(T, H, m.scales == "row", 1)
        with pytest.raises(ValueError, match="on a GPU"):
            m.forward((one.codes[0], one.scales[0]), w(T, E, dtype=F32), 2)


@pytest.mark.parametrize("kw", [
    dict(w13=None), dict(w2=None), dict(w13=w(E, 2 * I, H, dtype=F32)), dict(w13=w(2 * I, H)), dict(w2=w(E, H, I, dtype=F16)), dict(w2=w(E + 1, H, I)),
    dict(w2=w(E, H + 8, I)), dict(w2=w(E, H, I + 8)), dict(w13=w(E, 2 * I + 1, H)), dict(w13=w(E, 2 * I, H + 4)[:, :, :H]),
    dict(w13=w(E, H, 2 * I).transpose(1, 2)), dict(w13=w(0, 2 * I, H), w2=w(0, H, I)), dict(w13=w(1025, 8, 8), w2=w(1025, 8, 4)),
    dict(w13=w(E, 2 * I, 12), w2=w(E, 12, I)), dict(w13=w(E, 8, H), w2=w(E, H, 4)), dict(w2=f8(H, I)), dict(w13=f8(2 * I, H)),
    dict(w13=f8(2 * I, H), w2=f8(H, I, False)), dict(w13=f8(2 * I, H, False), w2=f8(H, I)), dict(w13=f8(16, H), w2=f8(H, 8)),
    dict(w13=f8(96, H, False), w2=f8(H, 48, False)), dict(w13=(w(E, 2 * I, H, dtype=U8), None), w2=f8(H, I)),
    dict(w13=f8(2 * I, H), w2=(f8(H, I)[0], w(E, H + 1, dtype=F32))), dict(act="tanh"), dict(act=1), dict(act=["silu"]), dict(bias13=w(E, I)),
    dict(bias13=w(E, 2 * I, dtype=torch.float64)), dict(bias2=w(H)), dict(bias2=[0.0])])
def test_layers_of_weights_that_do_not_fit(kw):
    with pytest.raises(ValueError):
        layer(**kw)


@pytest.mark.parametrize("w13,w2", [(None, w(E, H, I)), (w(2 * I, H), w(E, H, I)), (w(E, 2 * I, H), 3)])
def test_quantized_layers_of_what_is_no_weight(w13, w2):
    with pytest.raises(ValueError):
        X.ExpertsLayer.quantized(w13, w2)


@pytest.mark.parametrize("kw", [{}, dict(w13=f8(2 * I, H), w2=f8(H, I))])
@pytest.mark.parametrize("x,logits", [
    (w(T, H), w(T + 1, E, dtype=F32)), (w(T, H), w(T - 1, E, dtype=F32)), (w(T, H), w(T, E + 1, dtype=F32)), (w(T, H), w(T, E - 1, dtype=F32)),
    (w(T, H), None), (w(T, H), w(T * E, dtype=F32)), (None, w(T, E, dtype=F32)), (w(T, 1, H), w(T, E, dtype=F32)), ((), w(T, E, dtype=F32)),
    (w(1, H), w(T, E, dtype=F32)), ((w(T + 1, H, dtype=U8), w(T + 1, dtype=F32)), w(T, E, dtype=F32))])
def test_logits_of_other_tokens_or_experts(kw, x, logits):
    with pytest.raises(ValueError, match="^(?!.*on a GPU)"):
        layer(**kw).forward(x, logits, 2)
