"""The dense operators around the routed experts, as measured cases.

Three operators of ``nvfp4_w4a4_expert_amd.dense``:

  norm    s = x + residual; y = s / sqrt(mean(s^2) + eps) * (offset + weight);
          y rounded to x's type and/or held in 8 bits (E4M3 codes with one
          fp32 scale per row, or one power-of-two scale per 32 elements)
  quant   the same 8-bit forms of given rows (weights at load time, activations)
  linear  out = residual + act(a . w^T + bias), or act(gate) * up of a fused
          gate/up weight, on bf16, fp16 or 8-bit operands

``run`` computes them in plain torch operations (``own`` false) or with the
library's kernels (``own`` true).  Eight-bit codes are returned as
float8_e4m3fn tensors, power-of-two scales as float8_e8m0fnu tensors.
"""
import math

import torch

own = False

E4M3_MAX = 448.0
FLT_MAX = torch.finfo(torch.float32).max
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


# ---- the cases ---------------------------------------------------------------

def listed():
    return [
        # decode step of 16 tokens at the model's hidden size: residual added, the
        # experts' bf16 input and the dense half's 8-bit input in one call
        dict(name="norm_mx_decode", op="norm", t=16, h=2816, type="bf16", scales="mx", residual=True, y=True),
        # the same at an 8192-token prefill, with the new residual stream written
        dict(name="norm_mx_prefill", op="norm", t=8192, h=2816, type="bf16", scales="mx", residual=True, y=True),
        # fp16 rows of an expert's width, a ragged batch, 8-bit output alone with a scale per row
        dict(name="norm_row_fp16", op="norm", t=1237, h=704, type="fp16", scales="row", residual=False, y=False),
        # load time: the fused gate/up weight of a dense feed-forward, bf16 -> 8 bits
        dict(name="quant_mx_weight", op="quant", t=4224, h=2816, type="bf16", scales="mx"),
        # activations of a ragged fp16 batch, a scale per token
        dict(name="quant_row_fp16", op="quant", t=333, h=2112, type="fp16", scales="row"),
        # router logits (128 experts, fp32) of a decode batch and of a prefill
        dict(name="router_decode", op="linear", m=16, n=128, k=2816, type="bf16", act="none", gated=False, bias=False, residual=False, out="fp32"),
        dict(name="router_prefill", op="linear", m=4096, n=128, k=2816, type="bf16", act="none", gated=False, bias=False, residual=False, out="fp32"),
        # the dense feed-forward at prefill, 8 bits end to end: gate/up with its product
        # requantised in the epilogue, then down with the residual stream added
        dict(name="gate_up_mx", op="linear", m=4096, n=2112, k=2816, type="mx", act="gelu_tanh", gated=True, bias=False, residual=False, out="mx"),
        dict(name="down_mx", op="linear", m=4096, n=2816, k=2112, type="mx", act="none", gated=False, bias=False, residual=True, out="bf16"),
        # a ragged fp16 projection with bias and an odd number of outputs
        dict(name="bias_gelu_fp16", op="linear", m=1000, n=1411, k=704, type="fp16", act="gelu", gated=False, bias=True, residual=False, out="fp16"),
        # the largest: gate/up of an 8192-token prefill kept in bf16
        dict(name="gate_up_bf16", op="linear", m=8192, n=2112, k=2816, type="bf16", act="silu", gated=True, bias=False, residual=False, out="bf16"),
        # down projection of a few decoding tokens, a scale per row, bias and residual
        dict(name="down_row_decode", op="linear", m=5, n=2816, k=2112, type="row", act="none", gated=False, bias=True, residual=True, out="bf16"),
    ]


def _log(rng, lo, hi, step=1):
    """A multiple of `step` in [lo, hi], spread evenly over its logarithm."""
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return min(hi // step * step, max(-(-lo // step) * step, int(round(v / step)) * step))


def draw(rng):
    op = rng.choice(["norm", "quant", "linear", "linear"])
    if op in ("norm", "quant"):
        scales = rng.choice(["mx", "row", "none"] if op == "norm" else ["mx", "row"])
        h = _log(rng, 64, 8192, 32 if scales == "mx" else 8)
        t = _log(rng, 1, min(8192, max(1, 8192 * 2816 // h)))
        case = dict(op=op, t=t, h=h, type=rng.choice(["bf16", "fp16"]), scales=scales)
        if op == "norm":
            case.update(residual=rng.random() < 0.5, y=scales == "none" or rng.random() < 0.6)
        return case
    kind = rng.choice(["bf16", "fp16", "mx", "row"])
    out = rng.choice(["bf16", "fp16", "fp32", "mx"])
    gated = rng.random() < 0.35
    k = _log(rng, 64, 8192, 32 if kind == "mx" else 16 if kind == "row" else 8)
    n = _log(rng, 32, 8192, 32 if out == "mx" else 1)
    most = 8192 * 4224 * 2816 // (k * n * (2 if gated else 1))      # the largest listed product
    m = _log(rng, 1, max(1, min(8192, most)))
    return dict(op=op, m=m, n=n, k=k, type=kind, act=rng.choice(["none", "silu", "gelu", "gelu_tanh", "relu"]),
                gated=gated, bias=rng.random() < 0.5, residual=rng.random() < 0.5, out=out)


# ---- inputs ------------------------------------------------------------------

def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda")

    s = dict(case)
    if case["op"] in ("norm", "quant"):
        t, h, dt = case["t"], case["h"], TYPES[case["type"]]
        gain = torch.ones(h, device="cuda")
        gain[torch.rand(h, generator=g, device="cuda") < 0.01] = 30.0     # outlier channels
        x = normal(t, h) * gain
        if t > 4:
            x[t - 2] = 0.0                                               # a padding row
        s["x"] = x.to(dt)
        if case["op"] == "norm":
            r = normal(t, h) * 3.0
            if t > 4:
                r[t - 2] = 0.0
            s["r"] = r.to(dt) if case["residual"] else None
            s["weight"] = (0.2 * normal(h)).to(dt)
        return s
    m, n, k = case["m"], case["n"], case["k"]
    rows = 2 * n if case["gated"] else n
    a, w = normal(m, k), normal(rows, k) * (1.0 / math.sqrt(k))
    if case["type"] in ("mx", "row"):
        s["a"], s["w"] = (_to_bytes(_fp8(v, case["type"])) for v in (a, w))
    else:
        s["a"], s["w"] = a.to(TYPES[case["type"]]), w.to(TYPES[case["type"]])
    s["b"] = 0.5 * normal(rows) if case["bias"] else None
    s["r"] = normal(m, n).to(TYPES.get(case["out"], torch.bfloat16)) if case["residual"] else None
    return s


def _to_bytes(codes_scales):
    """(E4M3 codes, scales) as a program holds them: bytes, and bytes or fp32."""
    codes, scales = codes_scales
    return codes.view(torch.uint8), scales.view(torch.uint8) if scales.dtype != torch.float32 else scales


# ---- one pass ----------------------------------------------------------------

def run(s):
    if own:
        return _run_own(s)
    if s["op"] == "norm":
        return _norm(s)
    if s["op"] == "quant":
        codes, scales = _fp8(s["x"].float(), s["scales"])
        return {"codes": codes, "scales": scales}
    return _linear(s)


def _run_own(s):
    from nvfp4_w4a4_expert_amd import dense
    out = {}
    if s["op"] == "norm":
        y, total, fp8 = dense.rms_norm(s["x"], s["weight"], residual=s["r"], eps=1e-6, weight_offset=1.0,
                                       want_y=s["y"], scales=None if s["scales"] == "none" else s["scales"])
        if y is not None:
            out["y"] = y
        if s["r"] is not None:
            out["total"] = total
    elif s["op"] == "quant":
        fp8 = dense.quantize_fp8(s["x"], s["scales"])
    else:
        got = dense.linear(s["a"], s["w"], bias=s["b"], act=s["act"], gated=s["gated"], residual=s["r"],
                           out_dtype=TYPES.get(s["out"], "mx"))
        if s["out"] != "mx":
            return {"out": got}
        fp8 = got
    if fp8 is not None:
        out["codes"] = fp8.codes.view(torch.float8_e4m3fn)
        out["scales"] = fp8.scales if fp8.scales.dtype == torch.float32 else fp8.scales.view(torch.float8_e8m0fnu)
    return out


def _fp8(y, scales):
    """fp32 rows -> E4M3 codes with a scale amax/448 per row, or the smallest
    power of two that is no less than it per 32 elements."""
    t, h = y.shape
    if scales == "row":
        scale = y.abs().amax(1) / E4M3_MAX
        inv = torch.where(scale > 0, (1.0 / scale).clamp(max=FLT_MAX), torch.zeros_like(scale))
        return (y * inv[:, None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn), scale
    b = y.view(t, h // 32, 32)
    m, e = torch.frexp(b.abs().amax(2))                       # amax = m * 2^e, 448 = 0.875 * 2^9
    p = (e - 9 + (m > 0.875).to(e.dtype)).clamp(-126, 127)
    p = torch.where(m > 0, p, torch.full_like(p, -126))
    v = torch.ldexp(torch.ldexp(b, -(p // 2)[..., None]), -(p - p // 2)[..., None])
    codes = v.clamp(-E4M3_MAX, E4M3_MAX).view(t, h).to(torch.float8_e4m3fn)
    return codes, (p + 127).to(torch.uint8).view(torch.float8_e8m0fnu)


def _norm(s):
    x, out = s["x"], {}
    if s["r"] is not None:
        out["total"] = x = (x.float() + s["r"].float()).to(x.dtype)
    x = x.float()
    y = x * torch.rsqrt(x.square().mean(1, keepdim=True) + 1e-6) * (1.0 + s["weight"].float())
    if s["y"]:
        out["y"] = y.to(s["x"].dtype)
    if s["scales"] != "none":
        out["codes"], out["scales"] = _fp8(y, s["scales"])
    return out


def _values(v):
    """A linear operand in fp32."""
    if isinstance(v, torch.Tensor):
        return v.float()
    codes, scales = v
    y = codes.view(torch.float8_e4m3fn).float()
    if scales.dtype == torch.float32:
        return y * scales[:, None]
    return (y.view(y.shape[0], -1, 32) * scales.view(torch.float8_e8m0fnu).float()[..., None]).view(y.shape)


def _act(v, act):
    if act == "silu":
        return v * torch.sigmoid(v)
    if act == "gelu":
        return 0.5 * v * torch.erfc(v * -math.sqrt(0.5))
    if act == "gelu_tanh":
        return v * torch.sigmoid(math.sqrt(8 / math.pi) * (v + 0.044715 * v * v * v))
    return v.clamp(min=0.0) if act == "relu" else v


def _linear(s):
    v = _values(s["a"]) @ _values(s["w"]).t()
    if s["b"] is not None:
        v = v + s["b"]
    v = _act(v[:, :s["n"]], s["act"]) * v[:, s["n"]:] if s["gated"] else _act(v, s["act"])
    if s["r"] is not None:
        v = v + s["r"].float()
    if s["out"] == "mx":
        codes, scales = _fp8(v, "mx")
        return {"codes": codes, "scales": scales}
    return {"out": v.to(TYPES[s["out"]])}


# ---- what a pass cannot do without -------------------------------------------

def _row_bytes(h, kind):
    return {"bf16": 2 * h, "fp16": 2 * h, "fp32": 4 * h, "mx": h + h // 32, "row": h + 4, "none": 0}[kind]


def work(case):
    if case["op"] in ("norm", "quant"):
        t, h = case["t"], case["h"]
        each = 2 * h + _row_bytes(h, case["scales"])
        if case["op"] == "norm":
            each += (4 * h if case["residual"] else 0) + (2 * h if case["y"] else 0)
        return {"bytes": t * each + (2 * h if case["op"] == "norm" else 0), "flops": 6 * t * h}
    m, n, k = case["m"], case["n"], case["k"]
    rows = 2 * n if case["gated"] else n
    moved = (m + rows) * _row_bytes(k, case["type"]) + m * _row_bytes(n, case["out"])
    if case["residual"]:
        moved += m * _row_bytes(n, "bf16" if case["out"] == "mx" else case["out"])
    return {"bytes": moved + (4 * rows if case["bias"] else 0), "flops": 2 * m * rows * k}


# ---- the definition in 64 bits -----------------------------------------------

def exact(case, seed):
    """What `run` returns, in 64 bits, before the one rounding of each output
    (codes: the value that is rounded to E4M3).  The new residual stream and
    the scales are rounded by definition: later values are built on them."""
    s = prepare(case, seed)
    if case["op"] == "linear":
        a, w = _wide(s["a"]), _wide(s["w"])
        n = case["n"]
        gate = torch.mm(a, w[:n].t().contiguous())
        gate = gate if s["b"] is None else gate + s["b"][:n].double()
        v = _act_wide(gate, case["act"])
        if case["gated"]:
            up = torch.mm(a, w[n:].t().contiguous())
            v = v * (up if s["b"] is None else up + s["b"][n:].double())
        v = v if s["r"] is None else v + s["r"].double()
        return {"out": v} if case["out"] != "mx" else _wide_fp8(v, "mx")
    out, x = {}, s["x"].double()
    if case["op"] == "norm":
        if s["r"] is not None:
            x = (x + s["r"].double()).to(s["x"].dtype).double()
            out["total"] = x
        root = torch.sqrt(torch.linalg.vector_norm(x, dim=1).square() / case["h"] + 1e-6)
        x = x / root[:, None] * (s["weight"].double() + 1.0)
        if case["y"]:
            out["y"] = x
    if case["scales"] != "none":
        out.update(_wide_fp8(x, case["scales"]))
    return out


def _wide(v):
    if isinstance(v, torch.Tensor):
        return v.double()
    codes, scales = v
    if scales.dtype == torch.float32:
        return codes.view(torch.float8_e4m3fn).double() * scales.double().unsqueeze(1)
    step = torch.exp2(scales.double() - 127.0)
    return codes.view(torch.float8_e4m3fn).double() * step.repeat_interleave(32, dim=1)


def _act_wide(v, act):
    if act == "silu":
        return v / (1.0 + torch.exp(-v))
    if act == "gelu":
        return v * (1.0 + torch.erf(v / math.sqrt(2.0))) / 2.0
    if act == "gelu_tanh":
        return v * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (v + 0.044715 * v ** 3))) / 2.0
    return torch.relu(v) if act == "relu" else v


def _wide_fp8(v, scales):
    if scales == "row":
        scale = v.abs().max(dim=1).values / E4M3_MAX
        return {"codes": torch.where(scale[:, None] > 0, v / scale[:, None], torch.zeros_like(v)), "scales": scale}
    top = v.abs().reshape(v.shape[0], -1, 32).max(dim=2).values
    p = torch.floor(torch.log2(top.clamp(min=1e-300) / E4M3_MAX)) - 1.0
    for _ in range(3):                                        # up to the first power that covers the block
        p = torch.where(torch.exp2(p) * E4M3_MAX < top, p + 1.0, p)
    p = p.clamp(-126.0, 127.0)
    return {"codes": v / torch.exp2(p).repeat_interleave(32, dim=1), "scales": torch.exp2(p)}
