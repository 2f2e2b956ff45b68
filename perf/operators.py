"""The layer around the W4A4 product, measured: layer norm (forward, backward, and straight into the MXFP4
quantizer), the W4A4 product with bias, activation and residual in its epilogue, and that epilogue's backward.

Each operator is computed in a plain form from elementary torch operations (``own`` false) or by this
repository's kernels (``own`` true), on the same inputs. Formulas, per row x of X and with all arithmetic in
32 bits or more:

    norm        mu = mean(x), s = 1 / sqrt(mean((x - mu)^2) + eps), y = (x - mu) s w + b
    norm_grad   h = (x - mu) s, g = dy w, dx = s (g - mean(g) - h mean(g h)),
                dw = sum over rows of dy h, db = sum over rows of dy
    norm_quant  Q(y T): T block diagonal, K_j = G1 (x) ... (x) G5 per 32 channels, Q the MXFP4 quantizer
    linear      z = deq(A) deq(W)^T + bias, o = act(z) + residual
    linear_grad dz = do act'(z), dbias = sum over rows of dz
"""
import math

import torch

own = False

EPS = 1e-5
ACTS = ("none", "relu", "silu", "gelu", "gelu_tanh")
LEVELS = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def listed():
    return [
        # one token of a model of width 4096 being generated: latency
        {"name": "norm token", "op": "norm", "m": 1, "d": 4096, "type": "bf16"},
        # a whole prompt in front of a wide layer (8192 tokens x 4608 channels)
        {"name": "norm prompt", "op": "norm", "m": 8192, "d": 4608, "type": "bf16"},
        # a training step of a narrow model on 4096 tokens of 1152 channels
        {"name": "norm_grad narrow", "op": "norm_grad", "m": 4096, "d": 1152, "type": "bf16"},
        # the same with a 32-bit residual stream, a large batch of a wide model
        {"name": "norm_grad wide f32", "op": "norm_grad", "m": 16384, "d": 4096, "type": "f32"},
        # the quantized layer's input for one generated token
        {"name": "norm_quant token", "op": "norm_quant", "m": 1, "d": 4096, "type": "bf16", "packed": False},
        # the quantized layer's input for a prompt, scales laid out for the large product
        {"name": "norm_quant prompt", "op": "norm_quant", "m": 8192, "d": 4096, "type": "bf16", "packed": True},
        # one token through a down projection with its residual
        {"name": "linear token", "op": "linear", "m": 1, "n": 4096, "k": 4096, "type": "bf16", "act": "none",
         "bias": True, "residual": True, "pre": False, "packed": True},
        # a few dozen sequences generated together through an up projection whose width is no whole stage
        {"name": "linear batch", "op": "linear", "m": 45, "n": 4608, "k": 1152, "type": "bf16", "act": "silu",
         "bias": True, "residual": False, "pre": False, "packed": False},
        # a short prompt with ragged sizes, 32-bit outputs and residual stream
        {"name": "linear ragged f32", "op": "linear", "m": 509, "n": 1151, "k": 4608, "type": "f32", "act": "relu",
         "bias": True, "residual": True, "pre": False, "packed": False},
        # a training step's up projection, which keeps the values in front of the activation
        {"name": "linear train", "op": "linear", "m": 8192, "n": 16384, "k": 4096, "type": "bf16",
         "act": "gelu_tanh", "bias": True, "residual": False, "pre": True, "packed": True},
        # the backward of a short batch's epilogue in 32 bits, odd sizes
        {"name": "linear_grad odd f32", "op": "linear_grad", "m": 301, "n": 4607, "type": "f32", "act": "silu"},
        # the backward of the training step above
        {"name": "linear_grad train", "op": "linear_grad", "m": 8192, "n": 16384, "type": "bf16",
         "act": "gelu_tanh"},
    ]


def _size(rng, low, high, of=1):
    """A multiple of `of`, spread over the logarithm of low..high."""
    v = math.exp(rng.uniform(math.log(low), math.log(high + 1)))
    return max(of, min(high, int(v / of) * of))


def draw(rng):
    op = rng.choice(("norm", "norm_grad", "norm_quant", "linear", "linear", "linear_grad"))
    type_ = rng.choice(("bf16", "bf16", "f32"))
    if op in ("norm", "norm_grad"):
        d = _size(rng, 16, 16384, rng.choice((1, 8, 64)))
        return {"op": op, "m": _size(rng, 1, max(1, min(32768, (1 << 26) // d))), "d": d, "type": type_}
    if op == "norm_quant":
        packed = rng.random() < 0.5
        d = _size(rng, 256 if packed else 32, 16384, 256 if packed else 32)
        return {"op": op, "m": _size(rng, 1, max(1, min(16384, (1 << 25) // d))), "d": d, "type": type_,
                "packed": packed}
    act = rng.choice(ACTS)
    if op == "linear_grad":
        n = _size(rng, 16, 16384, rng.choice((1, 8)))
        return {"op": op, "m": _size(rng, 1, max(1, min(16384, (1 << 26) // n))), "n": n, "type": type_, "act": act}
    packed = rng.random() < 0.5
    k = _size(rng, 256 if packed else 32, 8192, 256 if packed else 32)
    n = _size(rng, 16, 16384, rng.choice((1, 16)))
    m = _size(rng, 1, max(1, min(8192, (1 << 38) // (n * k))))
    return {"op": op, "m": m, "n": n, "k": k, "type": type_, "act": act, "bias": rng.random() < 0.75,
            "residual": rng.random() < 0.5, "pre": rng.random() < 0.25, "packed": packed}


def work(case):
    m, t = case["m"], 2 if case["type"] == "bf16" else 4
    if case["op"] == "norm":
        d = case["d"]
        return {"bytes": 2 * m * d * t + 8 * d + 8 * m, "flops": 8 * m * d}
    if case["op"] == "norm_grad":
        d = case["d"]
        return {"bytes": 3 * m * d * t + 12 * d + 8 * m, "flops": 14 * m * d}
    if case["op"] == "norm_quant":
        d = case["d"]
        return {"bytes": m * d * t + m * d // 2 + m * d // 32 + 8 * d + 80 * (d // 32) + 8 * m, "flops": 20 * m * d}
    n = case["n"]
    if case["op"] == "linear_grad":
        return {"bytes": 3 * m * n * t + 4 * n, "flops": 10 * m * n}
    k = case["k"]
    operands = (m + n) * (k // 2 + k // 32) + 4 * n * case["bias"]
    return {"bytes": operands + m * n * t * (1 + case["residual"] + case["pre"]), "flops": 2 * m * n * k}


# ---------------------------------------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------------------------------------
def _type(case):
    return torch.bfloat16 if case["type"] == "bf16" else torch.float32


def _stream_values(g, m, d, dtype):
    """Activations of a residual stream: tokens and channels of unlike sizes, a few large channels, an offset."""
    x = torch.randn(m, d, generator=g, device="cuda")
    x *= 0.5 + 1.5 * torch.rand(m, 1, generator=g, device="cuda")
    x *= torch.exp(0.5 * torch.randn(d, generator=g, device="cuda"))
    large = torch.rand(d, generator=g, device="cuda") < 0.01
    x *= torch.where(large, 20.0, 1.0)
    return (x + 0.3 * torch.randn(d, generator=g, device="cuda")).to(dtype)


def _operand(g, rows, k, size):
    """An MXFP4 operand: codes [rows][k / 2] and E8M0 scales [rows][k / 32] of normal values."""
    v = torch.randn(rows, k, generator=g, device="cuda") * size
    v *= torch.exp(0.3 * torch.randn(k, generator=g, device="cuda"))
    index, e = _indices(v.view(rows, k // 32, 32))
    code = (index + 8 * torch.signbit(v).view(index.shape)).view(rows, k).to(torch.uint8)
    codes = code[:, 0::2] | (code[:, 1::2] << 4)
    return codes.contiguous(), (e + 127).view(rows, k // 32).to(torch.uint8)


def _pack(scales):
    """Scales [rows][k / 32] in the packed layout [k / 256][rows][8], even blocks of a stage first."""
    rows, blocks = scales.shape
    return scales.view(rows, blocks // 8, 4, 2).permute(1, 0, 3, 2).contiguous().view(blocks // 8, rows, 8)


def _unpack(packed):
    """The packed layout back as [rows][k / 32]."""
    stages, rows, _ = packed.shape
    return packed.view(stages, rows, 2, 4).permute(1, 0, 3, 2).reshape(rows, 8 * stages)


def prepare(case, seed):
    g = torch.Generator("cuda").manual_seed(seed)
    dtype, m, op = _type(case), case["m"], case["op"]
    s = {"case": dict(case)}
    if op in ("norm", "norm_grad", "norm_quant"):
        d = case["d"]
        s["x"] = _stream_values(g, m, d, dtype)
        s["weight"] = 1 + 0.2 * torch.randn(d, generator=g, device="cuda")
        s["bias"] = 0.1 * torch.randn(d, generator=g, device="cuda")
        if op == "norm_grad":
            s["dy"] = torch.randn(m, d, generator=g, device="cuda").to(dtype)
            x = s["x"].double()
            mu = x.mean(1, keepdim=True)
            s["mean"] = mu[:, 0].float()
            s["rstd"] = ((x - mu).square().mean(1) + EPS).rsqrt().float()
        if op == "norm_quant":
            # factors near the Hadamard start, as a calibration leaves them
            h = torch.tensor([[1.0, 1.0], [1.0, -1.0]], device="cuda") * 2 ** -0.5
            f = h + 0.1 * torch.randn(d // 32, 5, 2, 2, generator=g, device="cuda")
            s["factors"] = f.contiguous()
        return s
    n = case["n"]
    if op == "linear_grad":
        s["dout"] = torch.randn(m, n, generator=g, device="cuda").to(dtype)
        s["z"] = (1.5 * torch.randn(m, n, generator=g, device="cuda")).to(dtype)
        return s
    k = case["k"]
    s["codes_a"], sa = _operand(g, m, k, 1.0)
    s["codes_w"], sw = _operand(g, n, k, k ** -0.5)
    s["scales_a"], s["scales_w"] = (_pack(sa), _pack(sw)) if case["packed"] else (sa, sw)
    s["bias"] = 0.5 * torch.randn(n, generator=g, device="cuda") if case["bias"] else None
    s["residual"] = _stream_values(g, m, n, dtype) if case["residual"] else None
    return s


# ---------------------------------------------------------------------------------------------------------
# Plain forms
# ---------------------------------------------------------------------------------------------------------
def _indices(v):
    """Blocks of 32 values [..., 32]: the index of each one's E2M1 magnitude, ties to the even index, and the
    blocks' exponents (a zero block takes -127)."""
    top = v.abs().amax(-1, keepdim=True)
    e = (torch.frexp(top)[1] - 3).clamp(-127, 127)
    e = torch.where(top > 0, e, -127)
    u = torch.ldexp(v.abs(), -e)
    index = (u > 0.25).to(torch.int32)
    for border, even in ((0.75, True), (1.25, False), (1.75, True), (2.5, False), (3.5, True), (5.0, False)):
        index += (u >= border) if even else (u > border)
    return index, e


def _kronecker(f, dtype):
    """K [blocks][32][32] of factors [blocks][5][2][2]."""
    f = f.to(dtype)
    out = f[:, 0]
    for i in range(1, 5):
        n = out.shape[1]
        out = (out[:, :, None, :, None] * f[:, i][:, None, :, None, :]).reshape(-1, 2 * n, 2 * n)
    return out


def _decode(codes, scales, dtype):
    levels = torch.tensor(LEVELS + tuple(-v for v in LEVELS), dtype=dtype, device=codes.device)
    v = torch.stack((levels[(codes & 15).long()], levels[(codes >> 4).long()]), -1)
    rows, blocks = scales.shape
    return torch.ldexp(v.view(rows, blocks, 32), scales.to(torch.int32)[:, :, None] - 127).view(rows, 32 * blocks)


def _act(z, act):
    if act == "relu":
        return torch.where(z < 0, 0.0, z)
    if act == "silu":
        return z / (1 + torch.exp(-z))
    if act == "gelu":
        return 0.5 * z * (1 + torch.erf(z * 2 ** -0.5))
    if act == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh((2 / math.pi) ** 0.5 * (z + 0.044715 * z * z * z)))
    return z


def _act_grad(z, act):
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "silu":
        s = 1 / (1 + torch.exp(-z))
        return s * (1 + z * (1 - s))
    if act == "gelu":
        return 0.5 * (1 + torch.erf(z * 2 ** -0.5)) + z * torch.exp(-0.5 * z * z) * (2 * math.pi) ** -0.5
    if act == "gelu_tanh":
        c = (2 / math.pi) ** 0.5
        t = torch.tanh(c * (z + 0.044715 * z * z * z))
        return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * c * (1 + 3 * 0.044715 * z * z)
    return torch.ones_like(z)


def _plain(s):
    case = s["case"]
    op = case["op"]
    if op == "norm":
        x = s["x"].float()
        # the sum in 64 bits: a mean near zero is what is left of values that cancel
        mu = x.mean(1, keepdim=True, dtype=torch.float64).float()
        c = x - mu
        r = 1 / torch.sqrt((c * c).mean(1, keepdim=True) + EPS)
        return {"y": (c * r * s["weight"] + s["bias"]).to(s["x"].dtype), "mean": mu[:, 0], "rstd": r[:, 0]}
    if op == "norm_grad":
        dy, r = s["dy"].float(), s["rstd"][:, None]
        h = (s["x"].float() - s["mean"][:, None]) * r
        g = dy * s["weight"]
        dx = r * (g - g.mean(1, keepdim=True) - h * (g * h).mean(1, keepdim=True))
        return {"dx": dx.to(s["x"].dtype), "dweight": (dy * h).sum(0), "dbias": dy.sum(0)}
    if op == "norm_quant":
        # in 64 bits: next to a border between two codes the last bit of 32 decides
        x = s["x"].double()
        mu = x.mean(1, keepdim=True)
        c = x - mu
        r = 1 / torch.sqrt((c * c).mean(1, keepdim=True) + EPS)
        y = c * r * s["weight"] + s["bias"]
        m, d = y.shape
        k = _kronecker(s["factors"], y.dtype)
        t = torch.matmul(y.view(m, d // 32, 32).transpose(0, 1).contiguous(), k).transpose(0, 1)
        index, e = _indices(t)
        levels = torch.tensor(LEVELS, device=y.device)
        v = torch.ldexp(levels[index.long()], e)
        return {"values": torch.copysign(v, t.float()).reshape(m, d).to(torch.float8_e5m2),
                "mean": mu[:, 0].float(), "rstd": r[:, 0].float()}
    if op == "linear":
        sa, sw = s["scales_a"], s["scales_w"]
        if case["packed"]:
            sa, sw = _unpack(sa), _unpack(sw)
        z = torch.matmul(_decode(s["codes_a"], sa, torch.float32), _decode(s["codes_w"], sw, torch.float32).t())
        if s["bias"] is not None:
            z = z + s["bias"]
        o = _act(z, case["act"])
        if s["residual"] is not None:
            o = o + s["residual"].float()
        out = {"out": o.to(_type(case))}
        if case["pre"]:
            out["pre"] = z.to(_type(case))
        return out
    dz = s["dout"].float() * _act_grad(s["z"].float(), case["act"])
    return {"dz": dz.to(_type(case)), "dbias": dz.sum(0)}


def _framework(s):
    import mxfp4_activation_quantizer_amd as kq
    case = s["case"]
    op = case["op"]
    if op == "norm":
        y, mean, rstd = kq.layernorm(s["x"], s["weight"], s["bias"], eps=EPS, stats=True)
        return {"y": y, "mean": mean, "rstd": rstd}
    if op == "norm_grad":
        dx, dweight, dbias = kq.layernorm_backward(s["dy"], s["x"], s["mean"], s["rstd"], s["weight"])
        return {"dx": dx, "dweight": dweight, "dbias": dbias}
    if op == "norm_quant":
        codes, scales, mean, rstd = kq.layernorm_quantize_mxfp4(
            s["x"], s["weight"], s["bias"], s["factors"], eps=EPS, packed=case["packed"], stats=True)
        if case["packed"]:
            scales = _unpack(scales)
        # the codes as the values they stand for, in a type of 8 bits that holds them all
        return {"values": kq.dequantize_mxfp4_bf16(codes, scales).to(torch.float8_e5m2), "mean": mean, "rstd": rstd}
    if op == "linear":
        got = kq.mxfp4_linear(s["codes_a"], s["scales_a"], s["codes_w"], s["scales_w"], bias=s["bias"],
                              act=case["act"], residual=s["residual"], bf16=case["type"] == "bf16",
                              packed=case["packed"], want_pre=case["pre"])
        return {"out": got[0], "pre": got[1]} if case["pre"] else {"out": got}
    dz, dbias = kq.mxfp4_linear_backward(s["dout"], s["z"], act=case["act"])
    return {"dz": dz, "dbias": dbias}


def run(state):
    return _framework(state) if own else _plain(state)


# ---------------------------------------------------------------------------------------------------------
# The definitions in 64 bits
# ---------------------------------------------------------------------------------------------------------
def _exact_act(z, act):
    """(value, slope) of the activation at z."""
    one = torch.ones_like(z)
    if act == "relu":
        return z.clamp(min=0), torch.where(z > 0, one, 0 * one)
    if act == "silu":
        s = torch.sigmoid(z)
        return z * s, s + z * s * (1 - s)
    if act == "gelu":
        p = 0.5 * torch.erfc(-z / math.sqrt(2))
        return z * p, p + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    if act == "gelu_tanh":
        # (1 + tanh u) / 2 = sigmoid(2 u)
        c = math.sqrt(2 / math.pi)
        s = torch.sigmoid(2 * c * (z + 0.044715 * z ** 3))
        return z * s, s + z * s * (1 - s) * 2 * c * (1 + 0.134145 * z ** 2)
    return z, one


def exact(case, seed):
    s = prepare(case, seed)
    op, act = case["op"], case.get("act")
    if op in ("norm", "norm_quant"):
        x = s["x"].double()
        var, mean = torch.var_mean(x, 1, unbiased=False)
        rstd = (var + EPS) ** -0.5
        if op == "norm_quant":
            # the codes are steps of their inputs: next to a border no number of bits makes one side the right one
            return {"values": None, "mean": mean, "rstd": rstd}
        y = torch.addcmul(s["bias"].double(), (x - mean[:, None]) * rstd[:, None], s["weight"].double())
        return {"y": y, "mean": mean, "rstd": rstd}
    if op == "norm_grad":
        x, dy, w = s["x"].double(), s["dy"].double(), s["weight"].double()
        mean, rstd = s["mean"].double(), s["rstd"].double()
        h = (x - mean[:, None]) * rstd[:, None]
        a = torch.mv(dy, w) / x.shape[1]
        b = torch.mv(dy * h, w) / x.shape[1]
        return {"dx": (dy * w - a[:, None] - h * b[:, None]) * rstd[:, None], "dweight": (dy * h).sum(0),
                "dbias": dy.sum(0)}
    if op == "linear_grad":
        d = s["dout"].double() * _exact_act(s["z"].double(), act)[1]
        return {"dz": d, "dbias": d.sum(0)}
    # the codes by their bits: sign, two exponent bits of bias 1, one mantissa bit
    def value(codes, scales):
        c = torch.stack((codes & 15, codes >> 4), -1).flatten(1).int()
        ex, man = (c >> 1) & 3, (c & 1).double()
        mag = torch.where(ex > 0, (1 + man / 2) * 2.0 ** (ex - 1).double(), man / 2)
        return torch.where(c > 7, -mag, mag) * (2.0 ** (scales.double() - 127)).repeat_interleave(32, 1)

    sa, sw = (_unpack(s[n]) if case["packed"] else s[n] for n in ("scales_a", "scales_w"))
    z = value(s["codes_a"], sa) @ value(s["codes_w"], sw).T
    if s["bias"] is not None:
        z += s["bias"].double()
    o = _exact_act(z, act)[0]
    if s["residual"] is not None:
        o = o + s["residual"].double()
    return {"out": o, "pre": z} if case["pre"] else {"out": o}
