"""A layer's further operators around its experts, as measured cases.

Four operators of ``nvfp4_w4a4_expert_amd.dense`` and ``.experts``:

  block    b = x / sqrt(mean(x^2) + eps) * (offset + post_weight) (or x itself);
           total = residual_scale * residual + gate * b, rounded to x's type;
           y = total / sqrt(mean(total^2) + eps) * (offset + weight), rounded
           and/or held in 8 bits: a block's last norm, its gate, the residual
           stream's addition and the next block's first norm in one pass
  linear4  out = residual + act(a . w^T + bias), or act(gate) * up, with w held
           in 4 bits: E2M1 codes with an E4M3 scale per 16 elements and an fp32
           scale ("nv") or a power of two per 32 elements ("mx")
  grouped  the same product for rows grouped by expert, each group with its own
           weight: out[p] = act(a[row of p] . w[e]^T + bias[e]), groups of any
           size, none among them
  combine  out[t] = residual[t] + sum_j weights[t, j] * values[place of (t, j)]

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
EPS, RESIDUAL_SCALE = 1e-6, 0.8125


# ---- the cases ---------------------------------------------------------------

def listed():
    return [
        # decode step of 16 tokens at the model's hidden size: a learned gate per token
        # on the experts' output, the next block's bf16 and 8-bit inputs
        dict(name="block_decode", op="block", t=16, h=2816, type="bf16", post=True, gate="row", gate_act="sigmoid", scales="mx", y=True),
        # the same at an 8192-token prefill, with a gate per channel
        dict(name="block_prefill", op="block", t=8192, h=2816, type="bf16", post=True, gate="channel", gate_act="none", scales="mx", y=True),
        # one decoding token through the dense feed-forward's gate/up weight
        dict(name="w4_gate_up_token", op="linear4", m=1, n=2112, k=2816, type="bf16", scales="nv", act="gelu_tanh", gated=True, bias=False, residual=False, out="bf16"),
        # a decode batch on a large projection with power-of-two scales
        dict(name="w4_decode_mx", op="linear4", m=16, n=8192, k=8192, type="bf16", scales="mx", act="none", gated=False, bias=False, residual=True, out="bf16"),
        # a ragged fp16 batch of middle size with bias and an odd number of outputs
        dict(name="w4_ragged_fp16", op="linear4", m=77, n=1411, k=2112, type="fp16", scales="nv", act="silu", gated=False, bias=True, residual=False, out="fp16"),
        # the dense feed-forward's gate/up at prefill
        dict(name="w4_gate_up_prefill", op="linear4", m=4096, n=2112, k=2816, type="bf16", scales="nv", act="gelu_tanh", gated=True, bias=False, residual=False, out="bf16"),
        # decode step: 16 tokens, 8 of 128 experts each, gate/up: about a row per expert hit
        dict(name="experts_gate_up_decode", op="grouped", t=16, top=8, e=128, n=704, k=2816, type="bf16", act="silu", gated=True, bias=False, gather=True, out="bf16"),
        # a ragged fp16 batch on few experts, with bias and an odd number of outputs
        dict(name="experts_ragged_fp16", op="grouped", t=333, top=2, e=8, n=1411, k=704, type="fp16", act="gelu", gated=False, bias=True, gather=False, out="fp16"),
        # prefill of 4096 tokens: gate/up with the tokens gathered in the product
        dict(name="experts_gate_up_prefill", op="grouped", t=4096, top=8, e=128, n=704, k=2816, type="bf16", act="silu", gated=True, bias=False, gather=True, out="bf16"),
        # the down projection of the same rows, held in 8 bits
        dict(name="experts_down_mx", op="grouped", t=4096, top=8, e=128, n=2816, k=704, type="mx", act="none", gated=False, bias=False, gather=False, out="bf16"),
        # the experts' outputs back in token order: decode step in fp32, prefill in bf16
        dict(name="combine_decode", op="combine", t=16, top=8, h=2816, type="fp32", residual=True, out="bf16"),
        dict(name="combine_prefill", op="combine", t=4096, top=8, h=2816, type="bf16", residual=True, out="bf16"),
    ]


def _log(rng, lo, hi, step=1):
    """A multiple of `step` in [lo, hi], spread evenly over its logarithm."""
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return min(hi // step * step, max(-(-lo // step) * step, int(round(v / step)) * step))


def draw(rng):
    op = rng.choice(["block", "linear4", "linear4", "grouped", "grouped", "combine"])
    if op == "block":
        scales = rng.choice(["mx", "row", "none"])
        h = _log(rng, 64, 8192, 32 if scales == "mx" else 8)
        return dict(op=op, t=_log(rng, 1, min(8192, max(1, 8192 * 2816 // h))), h=h, type=rng.choice(["bf16", "fp16"]),
                    post=rng.random() < 0.7, gate=rng.choice(["none", "scalar", "row", "channel", "full"]),
                    gate_act=rng.choice(["none", "sigmoid", "tanh"]), scales=scales, y=scales == "none" or rng.random() < 0.6)
    act = rng.choice(["none", "silu", "gelu", "gelu_tanh", "relu"])
    gated, bias = rng.random() < 0.35, rng.random() < 0.5
    if op == "linear4":
        out = rng.choice(["bf16", "fp16", "fp32", "mx"])
        k = _log(rng, 64, 8192, 32)
        n = _log(rng, 32, 8192, 32 if out == "mx" else 1)
        most = 4096 * 4224 * 2816 // (k * n * (2 if gated else 1))         # the largest listed product
        return dict(op=op, m=_log(rng, 1, max(1, min(8192, most))), n=n, k=k, type=rng.choice(["bf16", "fp16"]),
                    scales=rng.choice(["nv", "mx"]), act=act, gated=gated, bias=bias, residual=rng.random() < 0.5, out=out)
    if op == "grouped":
        kind, out = rng.choice(["bf16", "fp16", "mx", "row"]), rng.choice(["bf16", "fp16", "fp32", "mx"])
        e = _log(rng, 2, 128)
        top = rng.randint(1, min(8, e))
        k = _log(rng, 64, 2816, 32 if kind == "mx" else 16 if kind == "row" else 8)
        n = _log(rng, 32, 2816 if not gated else 1408, 32 if out == "mx" else 1)
        n = min(n, 1408 * 2816 // (k * (2 if gated else 1)) // 32 * 32)    # the largest listed weights
        return dict(op=op, t=_log(rng, 1, max(1, min(8192, 4096 * 8 // top))), top=top, e=e, n=n, k=k, type=kind, act=act,
                    gated=gated, bias=bias, gather=rng.random() < 0.5, out=out)
    top, h = rng.randint(1, 8), _log(rng, 64, 8192, 8)
    return dict(op=op, t=_log(rng, 1, max(1, min(8192, 4096 * 8 * 2816 // (top * h)))), top=top, h=h,
                type=rng.choice(["bf16", "fp16", "fp32"]), residual=rng.random() < 0.5, out=rng.choice(["bf16", "fp16", "fp32"]))


# ---- inputs ------------------------------------------------------------------

def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda")

    s = dict(case)
    op, out = case["op"], TYPES.get(case.get("out"), torch.bfloat16)
    if op == "block":
        t, h, dt = case["t"], case["h"], TYPES[case["type"]]
        gain = torch.ones(h, device="cuda")
        gain[torch.rand(h, generator=g, device="cuda") < 0.01] = 30.0     # outlier channels
        x, r = normal(t, h) * gain, normal(t, h) * 3.0
        if t > 4:
            x[t - 2] = 0.0                                               # a padding row
            r[t - 2] = 0.0
        s["x"], s["r"] = x.to(dt), r.to(dt)
        s["w_post"] = (0.2 * normal(h)).to(dt) if case["post"] else None
        s["w"] = (0.2 * normal(h)).to(dt)
        shape = {"row": (t, 1), "channel": (h,), "full": (t, h)}.get(case["gate"])
        s["gate_at"] = 0.625 if case["gate"] == "scalar" else None if shape is None else normal(*shape).to(dt)
        return s
    if op == "combine":
        t, top, h = case["t"], case["top"], case["h"]
        s["values"] = normal(t * top, h).to(TYPES[case["type"]])
        s["weights"] = torch.softmax(normal(t, top), 1)
        s["inv"] = torch.randperm(t * top, generator=g, device="cuda").int()
        s["r"] = normal(t, h).to(out) if case["residual"] else None
        return s
    n, k = case["n"], case["k"]
    rows = 2 * n if case["gated"] else n
    if op == "linear4":
        s["a"] = normal(case["m"], k).to(TYPES[case["type"]])
        s["w"] = _fp4(normal(rows, k) * (1.0 / math.sqrt(k)), case["scales"])
        s["b"] = 0.5 * normal(rows) if case["bias"] else None
        s["r"] = normal(case["m"], n).to(out) if case["residual"] else None
        return s
    t, top, e = case["t"], case["top"], case["e"]
    # a router with experts that it likes and some that it hardly takes
    ids = torch.topk(normal(t, e) + 1.5 * normal(e), top, dim=1).indices
    order = torch.sort(ids.reshape(-1), stable=True).indices
    counts = torch.bincount(ids.reshape(-1), minlength=e)
    s["sizes"] = counts.tolist()                                         # (for the plain form's loop)
    s["offsets"] = torch.cat([counts.new_zeros(1), counts.cumsum(0)]).int()
    s["index"] = order.int() if case["gather"] else None
    a = normal(t if case["gather"] else t * top, k)
    scale = 1.0 / math.sqrt(k)
    if case["type"] in ("mx", "row"):
        s["a"] = _to_bytes(_fp8(a, case["type"]))
        each = [_to_bytes(_fp8(normal(rows, k) * scale, case["type"])) for _ in range(e)]
        s["w"] = tuple(torch.stack(v) for v in zip(*each))
    else:
        s["a"] = a.to(TYPES[case["type"]])
        s["w"] = torch.empty(e, rows, k, dtype=TYPES[case["type"]], device="cuda")
        for i in range(e):
            s["w"][i] = normal(rows, k) * scale
    s["b"] = 0.5 * normal(e, rows) if case["bias"] else None
    return s


def _to_bytes(codes_scales):
    """(E4M3 codes, scales) as a program holds them: bytes, and bytes or fp32."""
    codes, scales = codes_scales
    return codes.view(torch.uint8), scales.view(torch.uint8) if scales.dtype != torch.float32 else scales


def _fp4(w, scales):
    """fp32 rows -> (E2M1 codes two to a byte, block scales, fp32 scale or None)."""
    n, k = w.shape
    if scales == "nv":
        whole = (w.abs().max() / 2688.0).reshape(1)
        b = w.view(n, k // 16, 16)
        sf = (b.abs().amax(2) / 6.0 / whole).clamp(max=E4M3_MAX).to(torch.float8_e4m3fn)
        step = (sf.float() * whole)[..., None]
    else:
        whole = None
        b = w.view(n, k // 32, 32)
        sf = torch.ceil(torch.log2((b.abs().amax(2) / 6.0).clamp(min=2.0 ** -120))).to(torch.int32)
        step = torch.ldexp(torch.ones_like(b[..., :1]), sf[..., None])
        sf = (sf + 127).to(torch.uint8)
    v = torch.where(step > 0, b / step, torch.zeros_like(b)).view(n, k)
    borders = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=w.device)
    code = torch.bucketize(v.abs(), borders).to(torch.uint8) | ((v < 0).to(torch.uint8) << 3)
    return code[:, 0::2] | (code[:, 1::2] << 4), sf.view(torch.uint8), whole


# ---- one pass ----------------------------------------------------------------

def run(s):
    if own:
        return _run_own(s)
    return {"block": _block, "linear4": _linear4, "grouped": _grouped, "combine": _combine}[s["op"]](s)


def _run_own(s):
    from nvfp4_w4a4_expert_amd import dense, experts
    op, out = s["op"], {}
    if op == "combine":
        return {"out": experts.combine(s["values"], s["weights"], s["inv"], residual=s["r"], out_dtype=TYPES[s["out"]])}
    if op == "block":
        y, out["total"], fp8 = dense.block_norm(
            s["x"], s["r"], post_norm=s["post"], post_weight=s["w_post"], gate=s["gate_at"],
            gate_act=s["gate_act"] if isinstance(s["gate_at"], torch.Tensor) else None, residual_scale=RESIDUAL_SCALE,
            weight=s["w"], eps=EPS, weight_offset=1.0, want_y=s["y"], scales=None if s["scales"] == "none" else s["scales"])
        if y is not None:
            out["y"] = y
        if fp8 is None:
            return out
    else:
        kind = TYPES.get(s["out"], "mx")
        if op == "linear4":
            got = dense.linear(s["a"], dense.FP4Rows(*s["w"]), bias=s["b"], act=s["act"], gated=s["gated"],
                               residual=s["r"], out_dtype=kind)
        else:
            got = experts.grouped_linear(s["a"], s["w"], s["offsets"], index=s["index"], index_div=s["top"], bias=s["b"],
                                         act=s["act"], gated=s["gated"], out_dtype=kind)
        if kind != "mx":
            return {"out": got}
        fp8 = got
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


def _block(s):
    x, out = s["x"].float(), {}
    if s["post"]:
        x = x * torch.rsqrt(x.square().mean(1, keepdim=True) + EPS) * (1.0 + s["w_post"].float())
    gate = s["gate_at"]
    if isinstance(gate, torch.Tensor):
        gate = gate.float()
        gate = torch.sigmoid(gate) if s["gate_act"] == "sigmoid" else torch.tanh(gate) if s["gate_act"] == "tanh" else gate
    if gate is not None:
        x = x * gate
    out["total"] = (RESIDUAL_SCALE * s["r"].float() + x).to(s["x"].dtype)
    x = out["total"].float()
    y = x * torch.rsqrt(x.square().mean(1, keepdim=True) + EPS) * (1.0 + s["w"].float())
    if s["y"]:
        out["y"] = y.to(s["x"].dtype)
    if s["scales"] != "none":
        out["codes"], out["scales"] = _fp8(y, s["scales"])
    return out


def _act(v, act):
    if act == "silu":
        return v * torch.sigmoid(v)
    if act == "gelu":
        return 0.5 * v * torch.erfc(v * -math.sqrt(0.5))
    if act == "gelu_tanh":
        return v * torch.sigmoid(math.sqrt(8 / math.pi) * (v + 0.044715 * v * v * v))
    return v.clamp(min=0.0) if act == "relu" else v


def _epilogue(s, v, bias):
    if bias is not None:
        v = v + bias
    n = s["n"]
    return _act(v[:, :n], s["act"]) * v[:, n:] if s["gated"] else _act(v, s["act"])


def _stored(s, v):
    if s["out"] == "mx":
        codes, scales = _fp8(v, "mx")
        return {"codes": codes, "scales": scales}
    return {"out": v.to(TYPES[s["out"]])}


def _linear4(s):
    codes, sf, whole = s["w"]
    table = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0], device=codes.device)
    w = table[torch.stack([codes & 15, codes >> 4], 2).int()].view(codes.shape[0], -1)
    step = sf.view(torch.float8_e4m3fn).float() * whole if whole is not None else sf.view(torch.float8_e8m0fnu).float()
    w = (w.view(*sf.shape, -1) * step[..., None]).view(w.shape)
    v = _epilogue(s, s["a"].float() @ w.t(), s["b"])
    return _stored(s, v if s["r"] is None else v + s["r"].float())


def _values(v):
    """A grouped operand in fp32."""
    if isinstance(v, torch.Tensor):
        return v.float()
    codes, scales = v
    y = codes.view(torch.float8_e4m3fn).float()
    if scales.dtype == torch.float32:
        return y * scales[..., None]
    return (y.view(*scales.shape, 32) * scales.view(torch.float8_e8m0fnu).float()[..., None]).view(y.shape)


def _grouped(s):
    a = _values(s["a"])
    if s["index"] is not None:
        a = a[(s["index"] // s["top"]).long()]
    v = torch.empty(a.shape[0], s["n"], device=a.device)
    at = 0
    for e, size in enumerate(s["sizes"]):
        if size:
            w = _values(s["w"][e] if isinstance(s["w"], torch.Tensor) else (s["w"][0][e], s["w"][1][e]))
            v[at:at + size] = _epilogue(s, a[at:at + size] @ w.t(), None if s["b"] is None else s["b"][e])
            at += size
    return _stored(s, v)


def _combine(s):
    v = s["values"][s["inv"].long()].float().view(s["t"], s["top"], s["h"])
    v = (v * s["weights"][..., None]).sum(1)
    if s["r"] is not None:
        v = v + s["r"].float()
    return {"out": v.to(TYPES[s["out"]])}


# ---- what a pass cannot do without -------------------------------------------

def _row_bytes(h, kind):
    return {"bf16": 2 * h, "fp16": 2 * h, "fp32": 4 * h, "mx": h + h // 32, "row": h + 4, "none": 0}[kind]


def work(case):
    op = case["op"]
    if op == "block":
        t, h = case["t"], case["h"]
        each = 6 * h + _row_bytes(h, case["scales"]) + (2 * h if case["y"] else 0)
        gate = {"row": 2 * t, "channel": 2 * h, "full": 2 * t * h}.get(case["gate"], 0)
        return {"bytes": t * each + gate + 2 * h * (2 if case["post"] else 1), "flops": 14 * t * h}
    if op == "combine":
        t, top, h = case["t"], case["top"], case["h"]
        moved = t * top * (_row_bytes(h, case["type"]) + 8) + t * _row_bytes(h, case["out"]) * (2 if case["residual"] else 1)
        return {"bytes": moved, "flops": 2 * t * top * h}
    n, k = case["n"], case["k"]
    rows = 2 * n if case["gated"] else n
    if op == "linear4":
        m = case["m"]
        moved = m * _row_bytes(k, case["type"]) + rows * (k // 2 + k // (16 if case["scales"] == "nv" else 32)) + m * _row_bytes(n, case["out"])
        if case["residual"]:
            moved += m * _row_bytes(n, "bf16" if case["out"] == "mx" else case["out"])
        return {"bytes": moved + (4 * rows if case["bias"] else 0), "flops": 2 * m * rows * k}
    # weights of the experts that rows go to, as many as tokens of a router without likes would hit
    t, p, e = case["t"], case["t"] * case["top"], case["e"]
    hit = e * (1.0 - (1.0 - case["top"] / e) ** t)
    moved = (t if case["gather"] else p) * _row_bytes(k, case["type"]) + p * _row_bytes(n, case["out"])
    moved += int(hit * rows * (_row_bytes(k, case["type"]) + (4 if case["bias"] else 0)))
    return {"bytes": moved + (4 * p if case["gather"] else 0), "flops": 2 * p * rows * k}


# ---- the definition in 64 bits -----------------------------------------------

def exact(case, seed):
    """What `run` returns, in 64 bits, before the one rounding of each output
    (codes: the value that is rounded to E4M3).  The new residual stream and
    the scales are rounded by definition: later values are built on them."""
    s = prepare(case, seed)
    op = case["op"]
    if op == "block":
        return _wide_block(case, s)
    if op == "combine":
        t, top, h = case["t"], case["top"], case["h"]
        total = torch.zeros(t, h, dtype=torch.float64, device="cuda") if s["r"] is None else s["r"].double()
        place = s["inv"].long().reshape(t, top)
        for j in range(top):
            total += s["values"][place[:, j]].double() * s["weights"][:, j:j + 1].double()
        return {"out": total}
    if op == "linear4":
        codes, sf, whole = s["w"]
        low, high = codes.long() % 16, codes.long() // 16
        code = torch.stack((low, high), dim=-1).flatten(1)
        power, half = (code % 8) // 2, (code % 2).double()
        mag = torch.where(power == 0, half * 0.5, (1.0 + half * 0.5) * torch.exp2(power.double() - 1.0))
        w = torch.where(code >= 8, -mag, mag)
        each = case["k"] // sf.shape[1]
        if whole is None:
            w = w * torch.exp2(sf.double() - 127.0).repeat_interleave(each, dim=1)
        else:
            w = w * (sf.view(torch.float8_e4m3fn).double() * whole.double()).repeat_interleave(each, dim=1)
        v = _wide_product(case, s["a"].double(), w, s["b"])
        v = v if s["r"] is None else v + s["r"].double()
    else:
        v = torch.zeros(case["t"] * case["top"], case["n"], dtype=torch.float64, device="cuda")
        ends = s["offsets"].tolist()
        for e in range(case["e"]):
            lo, hi = ends[e], ends[e + 1]
            if lo == hi:
                continue
            take = torch.arange(lo, hi, device="cuda")
            if case["gather"]:
                take = torch.div(s["index"][lo:hi].long(), case["top"], rounding_mode="floor")
            if isinstance(s["a"], torch.Tensor):
                a, w = s["a"][take].double(), s["w"][e].double()
            else:
                a, w = (_wide(c, f) for c, f in ((s["a"][0][take], s["a"][1][take]), (s["w"][0][e], s["w"][1][e])))
            v[lo:hi] = _wide_product(case, a, w, None if s["b"] is None else s["b"][e])
    return {"out": v} if case["out"] != "mx" else _wide_fp8(v, "mx")


def _wide_product(case, a, w, bias):
    n = case["n"]
    gate = torch.mm(a, w[:n].t().contiguous())
    gate = gate if bias is None else gate + bias[:n].double()
    v = _act_wide(gate, case["act"])
    if case["gated"]:
        up = torch.mm(a, w[n:].t().contiguous())
        v = v * (up if bias is None else up + bias[n:].double())
    return v


def _wide_norm(x, weight):
    root = torch.sqrt(torch.linalg.vector_norm(x, dim=1).square() / x.shape[1] + EPS)
    return x / root[:, None] * (weight.double() + 1.0)


def _wide_block(case, s):
    b = _wide_norm(s["x"].double(), s["w_post"]) if case["post"] else s["x"].double()
    if case["gate"] != "none":
        gate = torch.as_tensor(s["gate_at"], device="cuda").double()
        if case["gate"] != "scalar" and case["gate_act"] != "none":
            gate = 1.0 / (1.0 + torch.exp(-gate)) if case["gate_act"] == "sigmoid" else 1.0 - 2.0 / (torch.exp(2.0 * gate) + 1.0)
        b = b * gate
    total = (s["r"].double() * RESIDUAL_SCALE + b).to(s["x"].dtype)
    out = {"total": total.double()}
    y = _wide_norm(total.double(), s["w"])
    if case["y"]:
        out["y"] = y
    if case["scales"] != "none":
        out.update(_wide_fp8(y, case["scales"]))
    return out


def _wide(codes, scales):
    v = codes.view(torch.float8_e4m3fn).double()
    if scales.dtype == torch.float32:
        return v * scales.double().unsqueeze(1)
    return v * torch.exp2(scales.double() - 127.0).repeat_interleave(32, dim=1)


def _act_wide(v, act):
    if act == "silu":
        return v / (1.0 + torch.exp(-v))
    if act == "gelu":
        return v * torch.special.erfc(v / -math.sqrt(2.0)) / 2.0
    if act == "gelu_tanh":
        return v / (1.0 + torch.exp(-2.0 * math.sqrt(2.0 / math.pi) * (v + 0.044715 * v ** 3)))
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
