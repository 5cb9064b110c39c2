"""Measured cases of the operators that run a feed-forward half of a transformer layer on
4-bit weights: the product of activations with a weight that qz_quantize left as MXFP4, NVFP4
or grouped INT4 (``linear``, ``linear_backward``), the gated feed-forward block on two such
weights (``gated_ffn``, ``gated_ffn_backward``) and the layer norm in front of them
(``layer_norm``, ``layer_norm_backward``).

``run`` computes each in its plain form (elementary torch operations in 32 bits, rounded once
at the end), or, where ``own`` is true, by the library's calls.  ``exact`` is the definition
in 64 bits.
"""
import math

import torch

own = False

BLOCK = {"mxfp4": 32, "nvfp4": 16}
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
EPS = 1e-5


def listed():
    return [
        # one token through a small projection: launch latency is all there is
        dict(name="linear 1 token small", op="linear", fmt="mxfp4", group=32, tokens=1, rows=1024, cols=1024, out="bf16"),
        # one decoded token through an attention-sized projection
        dict(name="linear 1 token nvfp4", op="linear", fmt="nvfp4", group=16, tokens=1, rows=4096, cols=4096, out="bf16"),
        # a short batch of decoded tokens through an output head, logits in fp32
        dict(name="linear 4 tokens logits", op="linear", fmt="mxfp4", group=32, tokens=4, rows=32768, cols=8192, out="f32"),
        # a small ragged decode batch, INT4 groups, an odd number of outputs
        dict(name="linear 7 tokens int4", op="linear", fmt="int4", group=128, tokens=7, rows=11001, cols=8192, out="bf16"),
        # the input gradient of a projection over a training batch
        dict(name="linear backward", op="linear_backward", fmt="nvfp4", group=16, tokens=2048, rows=8192, cols=4096),
        # one decoded token through the gated block
        dict(name="gated 1 token", op="gated_ffn", fmt="nvfp4", group=16, tokens=1, rows=16384, cols=4096, act="silu", save=False),
        # a ragged batch of decoded tokens, or a short prompt
        dict(name="gated 77 tokens", op="gated_ffn", fmt="mxfp4", group=32, tokens=77, rows=10240, cols=4096, act="silu", save=False),
        # a training batch, pre-activations kept for the backward pass
        dict(name="gated 4096 tokens", op="gated_ffn", fmt="nvfp4", group=16, tokens=4096, rows=16384, cols=4096, act="silu", save=True),
        # the backward pass of a short, odd batch
        dict(name="gated backward 131 tokens", op="gated_ffn_backward", fmt="mxfp4", group=32, tokens=131, rows=5632, cols=2048, act="gelu_tanh"),
        # the backward pass of the training batch
        dict(name="gated backward 4096 tokens", op="gated_ffn_backward", fmt="nvfp4", group=16, tokens=4096, rows=16384, cols=4096, act="silu"),
        # the norm of an activation-like tensor, tokens x hidden
        dict(name="norm 8192x4096", op="layer_norm", dtype="bf16", rows=8192, cols=4096),
        # its backward pass, with the weight's and the bias's gradient
        dict(name="norm backward 8192x4096", op="layer_norm_backward", dtype="bf16", rows=8192, cols=4096),
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["linear", "linear", "linear_backward", "gated_ffn", "gated_ffn_backward",
                     "layer_norm", "layer_norm_backward"])
    if op.startswith("layer_norm"):
        rows, cols = _spread(rng, 1, 16384), _spread(rng, 64, 16384)
        rows = max(1, min(rows, (8192 * 4096) // cols))
        return dict(op=op, dtype=rng.choice(["bf16", "bf16", "f32"]), rows=rows, cols=cols)
    fmt = rng.choice(["mxfp4", "nvfp4", "int4"])
    group = BLOCK.get(fmt) or rng.choice([32, 64, 128])
    tokens, rows, cols = _spread(rng, 1, 4096), _spread(rng, 512, 32768), _spread(rng, 512, 8192)
    unit = max(group, 32)
    cols = max(unit, cols // unit * unit)
    two = 2 if op.startswith("gated") else 1
    if op == "linear":
        rows |= rng.choice([0, 1])  # an odd number of outputs now and then
    else:
        rows = max(8, min(rows, 16384) // 8 * 8)
    tokens = max(1, min(tokens, (4096 * 32768 * 4096) // (two * rows * cols)))
    case = dict(op=op, fmt=fmt, group=group, tokens=tokens, rows=rows, cols=cols)
    if op == "linear":
        case["out"] = rng.choice(["bf16", "bf16", "f32"])
    if op.startswith("gated"):
        case["act"] = rng.choice(["silu", "gelu_tanh"])
    if op == "gated_ffn":
        case["save"] = rng.choice([False, True])
    return case


# ---- inputs ---------------------------------------------------------------------------------
def _weight(fmt, group, rows, cols, gen):
    """A weight-like [rows, cols] tensor in the library's 4-bit layouts: N(0, 0.02^2) with 0.1 %
    of the values 10 times as large; codes (two a byte, the first in the low nibble), scales
    and, for NVFP4, the tensor scale."""
    dev = gen.device
    codes = torch.empty(rows, cols // 2, dtype=torch.uint8, device=dev)
    scales = torch.empty(rows, cols // group, device=dev,
                         dtype=torch.float32 if fmt == "int4" else torch.uint8)
    tensor = torch.full((1,), 1.0, dtype=torch.float32, device=dev)
    if fmt == "nvfp4":
        tensor.fill_(1.25 / 2688.0)
    mid = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=dev)
    step = max(1, (1 << 25) // cols)
    for r0 in range(0, rows, step):
        n = min(step, rows - r0)
        w = torch.randn(n, cols, device=dev, generator=gen) * 0.02
        w *= 1 + 9 * (torch.rand(n, cols, device=dev, generator=gen) < 1e-3)
        w = w.reshape(n, cols // group, group)
        a = w.abs().amax(-1, keepdim=True)
        if fmt == "int4":
            s = a / 7
            q = (w / s).round().clamp(-7, 7).to(torch.int8)
            c = (q & 15).to(torch.uint8).reshape(n, cols)
            scales[r0:r0 + n] = s[..., 0]
        else:
            if fmt == "mxfp4":
                k = torch.ceil(torch.log2(a / 6))
                s = torch.exp2(k)
                scales[r0:r0 + n] = (k[..., 0] + 127).to(torch.uint8)
            else:
                e4 = (a / 6 / tensor).clamp(2.0 ** -9, 448).to(torch.float8_e4m3fn)
                s = e4.float() * tensor
                scales[r0:r0 + n] = e4.view(torch.uint8)[..., 0]
            v = w / s
            c = torch.bucketize(v.abs(), mid).to(torch.uint8) + 8 * (v < 0).to(torch.uint8)
            c = c.reshape(n, cols)
        codes[r0:r0 + n] = c[:, 0::2] | (c[:, 1::2] << 4)
    return codes, scales, tensor


def _activations(tokens, cols, gen):
    """Normalised hidden states, [tokens, cols] bf16: N(0, 1) with 8 outlier channels."""
    x = torch.randn(tokens, cols, device=gen.device, generator=gen)
    at = torch.randint(0, cols, (8,), device=gen.device, generator=gen)
    x[:, at] *= 20 + 40 * torch.rand(8, device=gen.device, generator=gen)
    return x.to(torch.bfloat16)


def _inputs(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))

    def normal(*shape):
        return torch.randn(*shape, device="cuda", generator=gen)

    op, s = case["op"], dict(case)
    if op.startswith("layer_norm"):
        dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
        rows, cols = case["rows"], case["cols"]
        x = normal(rows, cols) + 0.5 * normal(1, cols)
        s["x"] = x.to(dt)
        s["weight"], s["bias"] = 1 + 0.1 * normal(cols), 0.1 * normal(cols)
        if op == "layer_norm_backward":
            s["dy"] = (normal(rows, cols) * 0.01).to(dt)
            x = s["x"].float()
            s["mean"] = x.mean(-1)
            s["rstd"] = torch.rsqrt((x - s["mean"][:, None]).square().mean(-1) + EPS)
        return s
    tokens, rows, cols = case["tokens"], case["rows"], case["cols"]
    s["w0"] = _weight(case["fmt"], case["group"], rows, cols, gen)
    if op.startswith("gated"):
        s["w1"] = _weight(case["fmt"], case["group"], rows, cols, gen)
    if op in ("linear", "gated_ffn"):
        s["x"] = _activations(tokens, cols, gen)
    else:
        s["dy"] = (normal(tokens, rows) * 0.01).to(torch.bfloat16)
    if op == "gated_ffn_backward":
        s["g"], s["u"] = ((1.5 * normal(tokens, rows)).to(torch.bfloat16) for _ in range(2))
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    if own and "w0" in s:  # the handles that a program keeps with its quantized weights
        import precision_quantization_gb300 as qz
        fmt = qz.FORMATS[case["fmt"]]
        for k in ("w0", "w1"):
            if k in s:
                codes, scales, tensor = s[k]
                s[k] = qz.Weight(qz.Quantized(codes, scales, tensor, fmt, qz.QZ_GRAN_BLOCK,
                                              qz.QZ_SCALE_UP, case["rows"], case["cols"],
                                              case["group"]))
    return s


# ---- one pass ---------------------------------------------------------------------------------
def _run_own(s):
    import precision_quantization_gb300 as qz
    op = s["op"]
    if op == "linear":
        return qz.linear(s["x"], s["w0"], out_dtype=torch.float32 if s["out"] == "f32" else torch.bfloat16)
    if op == "linear_backward":
        return qz.linear_backward(s["dy"], s["w0"])
    if op == "gated_ffn":
        return qz.gated_ffn(s["x"], s["w0"], s["w1"], activation=s["act"], save=s["save"])
    if op == "gated_ffn_backward":
        return qz.gated_ffn_backward(s["dy"], s["g"], s["u"], s["w0"], s["w1"], activation=s["act"])
    if op == "layer_norm":
        return qz.layer_norm(s["x"], s["weight"], s["bias"], eps=EPS)
    return qz.layer_norm_backward(s["dy"], s["x"], s["mean"], s["rstd"], s["weight"])


def _dequantize(s, w):
    codes, scales, tensor = w
    rows, cols, group = s["rows"], s["cols"], s["group"]
    c = torch.stack((codes & 15, codes >> 4), -1).reshape(rows, cols)
    if s["fmt"] == "int4":
        v = ((c ^ 8).to(torch.int8) - 8).float()
        k = scales
    else:
        table = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=codes.device)
        v = table[c.int()]
        k = torch.exp2(scales.float() - 127) if s["fmt"] == "mxfp4" else scales.view(torch.float8_e4m3fn).float() * tensor
    return (v.reshape(rows, -1, group) * k[..., None]).reshape(rows, cols)


def _act(g, act):
    if act == "silu":
        return g / (1 + torch.exp(-g))
    return 0.5 * g * (1 + torch.tanh(math.sqrt(2 / math.pi) * (g + 0.044715 * g * g * g)))


def _act_grad(g, act):
    if act == "silu":
        p = 1 / (1 + torch.exp(-g))
        return p * (1 + g * (1 - p))
    c = math.sqrt(2 / math.pi)
    t = torch.tanh(c * (g + 0.044715 * g * g * g))
    return 0.5 * (1 + t) + 0.5 * g * (1 - t * t) * c * (1 + 3 * 0.044715 * g * g)


def run(s):
    if own:
        return _run_own(s)
    op, bf = s["op"], torch.bfloat16
    if op == "linear":
        return (s["x"].float() @ _dequantize(s, s["w0"]).T).to(torch.float32 if s["out"] == "f32" else bf)
    if op == "linear_backward":
        return (s["dy"].float() @ _dequantize(s, s["w0"])).to(bf)
    if op == "gated_ffn":
        x = s["x"].float()
        g = x @ _dequantize(s, s["w0"]).T
        u = x @ _dequantize(s, s["w1"]).T
        h = _act(g, s["act"]) * u
        return (h.to(bf), g.to(bf), u.to(bf)) if s["save"] else h.to(bf)
    if op == "gated_ffn_backward":
        dh, g, u = s["dy"].float(), s["g"].float(), s["u"].float()
        dg, du = dh * u * _act_grad(g, s["act"]), dh * _act(g, s["act"])
        dx = dg @ _dequantize(s, s["w0"]) + du @ _dequantize(s, s["w1"])
        return dx.to(bf), dg.to(bf), du.to(bf)
    x = s["x"].float()
    if op == "layer_norm":
        mean = x.mean(-1)
        d = x - mean[:, None]
        rstd = torch.rsqrt((d * d).mean(-1) + EPS)
        return (d * rstd[:, None] * s["weight"] + s["bias"]).to(s["x"].dtype), mean, rstd
    dy = s["dy"].float()
    n = (x - s["mean"][:, None]) * s["rstd"][:, None]
    t = dy * s["weight"]
    dx = s["rstd"][:, None] * (t - t.mean(-1, keepdim=True) - n * (t * n).mean(-1, keepdim=True))
    return dx.to(s["x"].dtype), (dy * n).sum(0), dy.sum(0)


def work(case):
    op = case["op"]
    if op.startswith("layer_norm"):
        n, e = case["rows"] * case["cols"], 2 if case["dtype"] == "bf16" else 4
        if op == "layer_norm":
            return {"bytes": 2 * n * e + 8 * case["rows"] + 8 * case["cols"], "flops": 8 * n}
        return {"bytes": 3 * n * e + 8 * case["rows"] + 12 * case["cols"], "flops": 14 * n}
    tokens, rows, cols = case["tokens"], case["rows"], case["cols"]
    two = 2 if op.startswith("gated") else 1
    weights = two * (rows * cols // 2 + rows * cols // case["group"] * (4 if case["fmt"] == "int4" else 1))
    acts = {"linear": cols * 2 + rows * (4 if case.get("out") == "f32" else 2),
            "linear_backward": (cols + rows) * 2,
            "gated_ffn": cols * 2 + rows * (6 if case.get("save") else 2),
            "gated_ffn_backward": rows * 10 + cols * 2}[op]
    return {"bytes": weights + tokens * acts, "flops": 2 * two * tokens * rows * cols}


# ---- the definition in 64 bits ------------------------------------------------------------------
def _values64(case, w):
    """The weight's values from its fields: sign, exponent and mantissa bits of each code."""
    codes, scales, tensor = w
    rows, cols = case["rows"], case["cols"]
    out = torch.empty(rows, cols, dtype=torch.float64, device=codes.device)
    for half, nibble in ((0, codes % 16), (1, codes // 16)):
        c = nibble.to(torch.int64)
        if case["fmt"] == "int4":
            v = torch.where(c >= 8, c - 16, c).double()
        else:
            e, m = (c >> 1) & 3, (c & 1).double()
            v = torch.where(e > 0, torch.ldexp(1 + m / 2, (e - 1).double()), m / 2)
            v = torch.where(c >= 8, -v, v)
        out[:, half::2] = v
    if case["fmt"] == "int4":
        k = scales.double()
    else:
        b = scales.to(torch.int64)
        if case["fmt"] == "mxfp4":
            k = torch.ldexp(torch.ones_like(b, dtype=torch.float64), (b - 127).double())
        else:
            e, m = (b >> 3) & 15, (b & 7).double()
            k = torch.where(e > 0, torch.ldexp(1 + m / 8, (e - 7).double()), m / 512) * tensor.double()
    return out.mul_(k.repeat_interleave(case["group"], 1))


def _act64(g, act):
    """The activation and its derivative."""
    if act == "silu":
        p = torch.sigmoid(g)
        return g * p, p + g * p * (1 - p)
    a, b = math.sqrt(2 / math.pi), 0.044715
    e = torch.exp(-2 * a * (g + b * g ** 3))  # (1 + tanh z) / 2 = 1 / (1 + exp(-2 z))
    p = 1 / (1 + e)
    return g * p, p + g * p * (1 - p) * 2 * a * (1 + 3 * b * g * g)


def exact(case, seed):
    s, op = _inputs(case, seed), case["op"]
    if op.startswith("layer_norm"):
        x, w = s["x"].double(), s["weight"].double()
        if op == "layer_norm":
            var, mean = torch.var_mean(x, -1, correction=0)
            rstd = 1 / torch.sqrt(var + EPS)
            return torch.addcmul(s["bias"].double(), (x - mean[:, None]) * rstd[:, None], w), mean, rstd
        dy, rstd = s["dy"].double(), s["rstd"].double()[:, None]
        n = x.sub(s["mean"].double()[:, None]).mul(rstd)
        t = dy * w
        a, b = torch.einsum("rc->r", t) / x.shape[1], torch.einsum("rc,rc->r", t, n) / x.shape[1]
        return (t - a[:, None] - n * b[:, None]) * rstd, torch.einsum("rc,rc->c", dy, n), torch.einsum("rc->c", dy)
    w0 = _values64(case, s["w0"])
    if op == "linear":
        return torch.einsum("tc,rc->tr", s["x"].double(), w0)
    if op == "linear_backward":
        return torch.einsum("tr,rc->tc", s["dy"].double(), w0)
    w1 = _values64(case, s["w1"])
    if op == "gated_ffn":
        g, u = torch.einsum("tc,rc->tr", s["x"].double(), w0), torch.einsum("tc,rc->tr", s["x"].double(), w1)
        h = _act64(g, case["act"])[0].mul_(u)
        return (h, g, u) if case["save"] else h
    a, da = _act64(s["g"].double(), case["act"])
    dg, du = s["dy"].double() * s["u"].double() * da, s["dy"].double() * a
    return torch.einsum("tr,rc->tc", dg, w0) + torch.einsum("tr,rc->tc", du, w1), dg, du
