"""What a transformer block needs between its W4A4 products, measured: the gated feed-forward product (forward and
the backward of its epilogue), the norm of each query and key head with the position rotation in the same pass
(forward and backward), and a cache of keys and values in MXFP4, quantized as it is written and read back.

Each operator is computed in a plain form from elementary torch operations (``own`` false) or by this
repository's kernels (``own`` true), on the same inputs. Formulas, with all arithmetic in 32 bits or more:

    gated       g = deq(A) deq(Wg)^T + bg, u = deq(A) deq(Wu)^T + bu, o = act(g) u
    gated_grad  dg = do u act'(g), du = do act(g), dbg and dbu their sums over the rows
    head        per head x of a token: s = 1 / sqrt(mean(x^2) + eps), n = x s w (w one of two, for query heads and
                for key heads), then the first r channels of n in pairs (a, b) of angle t = p f_i, p the token's position:
                (a cos t - b sin t, b cos t + a sin t) times an amplitude; pairs (i, i + r / 2) or (2 i, 2 i + 1)
    head_grad   e the rotated-back and amplified dy, h = x s: dx = s (e w - h mean(e w h)),
                dw = sum of e h over the tokens and the heads of that weight
    cache_write row slots[i] of the caches = Q(head(k_i)), Q(v_i), Q the MXFP4 quantizer
    cache_read  deq of the rows slots[i]
"""
import math

import torch

own = False

EPS = 1e-6
ACTS = ("none", "relu", "silu", "gelu", "gelu_tanh")
LEVELS = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def listed():
    return [
        # one token being generated: the two projections of its feed-forward block
        {"name": "gated token", "op": "gated", "m": 1, "n": 11008, "k": 4096, "type": "bf16", "act": "silu",
         "bias": False, "pre": False, "packed": True},
        # the same for a batch of prompts
        {"name": "gated prompt", "op": "gated", "m": 8192, "n": 11008, "k": 4096, "type": "bf16", "act": "silu",
         "bias": False, "pre": False, "packed": True},
        # the backward of a short batch in 32 bits, odd sizes
        {"name": "gated_grad odd f32", "op": "gated_grad", "m": 301, "n": 4607, "type": "f32", "act": "gelu"},
        # the backward of a training step
        {"name": "gated_grad train", "op": "gated_grad", "m": 8192, "n": 11008, "type": "bf16", "act": "silu"},
        # one token being generated, far into its context: 32 query heads that share 8 key heads
        {"name": "head token", "op": "head", "m": 1, "q": 32, "k": 8, "d": 128, "rot": 128, "inter": False,
         "axes": 1, "start": 131000, "type": "bf16"},
        # a prompt of the same
        {"name": "head prompt", "op": "head", "m": 8192, "q": 32, "k": 8, "d": 128, "rot": 128, "inter": False,
         "axes": 1, "start": 0, "type": "bf16"},
        # an image of 64 x 64 tokens in training: 1152 channels in 16 heads, a position for each of its two axes, in 32 bits
        {"name": "head_grad image f32", "op": "head_grad", "m": 4096, "q": 16, "k": 16, "d": 72, "rot": 72,
         "inter": True, "axes": 2, "start": 0, "type": "f32"},
        # a training step on 8192 tokens
        {"name": "head_grad train", "op": "head_grad", "m": 8192, "q": 32, "k": 8, "d": 128, "rot": 128,
         "inter": False, "axes": 1, "start": 0, "type": "bf16"},
        # 64 sequences generated together: one key and value row of each into its page
        {"name": "cache_write batch", "op": "cache_write", "m": 64, "h": 8, "d": 128, "rot": 128, "inter": False,
         "norm": True, "start": 2000, "type": "bf16"},
        # a prompt into the cache
        {"name": "cache_write prompt", "op": "cache_write", "m": 8192, "h": 8, "d": 128, "rot": 128, "inter": False,
         "norm": True, "start": 0, "type": "bf16"},
        # a short cached prefix in front of a new turn
        {"name": "cache_read prefix", "op": "cache_read", "m": 509, "h": 8, "d": 128, "type": "bf16"},
        # a long context read back for the next piece of its prompt
        {"name": "cache_read context", "op": "cache_read", "m": 131072, "h": 8, "d": 128, "type": "bf16"},
    ]


def _size(rng, low, high, of=1):
    """A multiple of `of`, spread over the logarithm of low..high."""
    v = math.exp(rng.uniform(math.log(low), math.log(high + 1)))
    return max(of, min(high, int(v / of) * of))


def draw(rng):
    op = rng.choice(("gated", "gated", "gated_grad", "head", "head_grad", "cache_write", "cache_read"))
    type_ = rng.choice(("bf16", "bf16", "f32"))
    act = rng.choice(ACTS)
    if op == "gated":
        packed = rng.random() < 0.5
        k = _size(rng, 256 if packed else 32, 8192, 256 if packed else 32)
        n = _size(rng, 16, 11008, rng.choice((1, 16)))
        m = _size(rng, 1, max(1, min(8192, (1 << 37) // (n * k))))
        return {"op": op, "m": m, "n": n, "k": k, "type": type_, "act": act, "bias": rng.random() < 0.5,
                "pre": rng.random() < 0.25, "packed": packed}
    if op == "gated_grad":
        n = _size(rng, 16, 11008, rng.choice((1, 8)))
        return {"op": op, "m": _size(rng, 1, max(1, min(8192, (1 << 25) // n))), "n": n, "type": type_, "act": act}
    if op == "cache_read":
        h, d = rng.choice((1, 2, 4, 5, 8, 16)), rng.choice((32, 64, 96, 128, 160, 256))
        return {"op": op, "m": _size(rng, 1, (1 << 26) // (h * d)), "h": h, "d": d, "type": type_}
    if op == "cache_write":
        h, d = rng.choice((1, 2, 4, 5, 8, 16)), rng.choice((32, 64, 96, 128, 160, 256))
        return {"op": op, "m": _size(rng, 1, min(8192, (1 << 23) // (h * d))), "h": h, "d": d,
                "rot": rng.choice((0, d // 2, d, d)), "inter": rng.random() < 0.5, "norm": rng.random() < 0.7,
                "start": _size(rng, 1, 200000), "type": type_}
    d = rng.choice((32, 40, 64, 72, 80, 96, 128, 128, 160, 192, 256, 512, 65))
    k = rng.choice((1, 2, 4, 5, 8, 16))
    rot = rng.choice((0, d // 4 * 2, d // 2 * 2, d // 2 * 2))
    q = k * rng.choice((1, 1, 2, 4, 7))
    return {"op": op, "m": _size(rng, 1, max(1, min(8192, (1 << 24) // ((q + k) * d)))), "q": q, "k": k, "d": d,
            "rot": rot, "inter": rng.random() < 0.5, "axes": rng.choice((1, 1, 2, 3)) if rot >= 6 else 1,
            "start": _size(rng, 1, 200000), "type": type_}


def work(case):
    m, t, op = case["m"], 2 if case["type"] == "bf16" else 4, case["op"]
    if op == "gated":
        n, k = case["n"], case["k"]
        return {"bytes": (m + 2 * n) * (k // 2 + k // 32) + 8 * n * case["bias"] + m * n * t * (1 + 2 * case["pre"]),
                "flops": 4 * m * n * k}
    if op == "gated_grad":
        n = case["n"]
        return {"bytes": 5 * m * n * t + 8 * n, "flops": 15 * m * n}
    d = case["d"]
    if op == "cache_read":
        return {"bytes": m * case["h"] * (d // 2 + d // 32 + d * t) + 8 * m, "flops": 2 * m * case["h"] * d}
    if op == "cache_write":
        return {"bytes": 2 * m * case["h"] * (d // 2 + d // 32 + d * t) + 16 * m + 4 * d * case["norm"] + 4 * case["rot"],
                "flops": 12 * m * case["h"] * d}
    h = case["q"] + case["k"]
    tables = 8 * m * case["axes"] + 4 * case["rot"] + 8 * d
    if op == "head":
        return {"bytes": 2 * m * h * d * t + tables, "flops": 8 * m * h * d}
    return {"bytes": 3 * m * h * d * t + tables + 8 * d, "flops": 18 * m * h * d}


# ---------------------------------------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------------------------------------
def _type(case):
    return torch.bfloat16 if case["type"] == "bf16" else torch.float32


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


def _operand(g, rows, k, size):
    """An MXFP4 operand: codes [rows][k / 2] and E8M0 scales [rows][k / 32] of normal values."""
    v = torch.randn(rows, k, generator=g, device="cuda") * size
    v *= torch.exp(0.3 * torch.randn(k, generator=g, device="cuda"))
    index, e = _indices(v.view(rows, k // 32, 32))
    code = (index + 8 * torch.signbit(v).view(index.shape)).view(rows, k).to(torch.uint8)
    return (code[:, 0::2] | (code[:, 1::2] << 4)).contiguous(), (e + 127).view(rows, k // 32).to(torch.uint8)


def _pack(scales):
    """Scales [rows][k / 32] in the packed layout [k / 256][rows][8], even blocks of a stage first."""
    rows, blocks = scales.shape
    return scales.view(rows, blocks // 8, 4, 2).permute(1, 0, 3, 2).contiguous().view(blocks // 8, rows, 8)


def _unpack(packed):
    """The packed layout back as [rows][k / 32]."""
    stages, rows, _ = packed.shape
    return packed.view(stages, rows, 2, 4).permute(1, 0, 3, 2).reshape(rows, 8 * stages)


def _axis_pairs(case):
    """How many of the rotated pairs take their angle from each axis of the position."""
    n, axes = case["rot"] // 2, case.get("axes", 1)
    return [n // axes + (1 if i < n % axes else 0) for i in range(axes)]


def _positions(case, g):
    """One axis: the tokens follow each other from the start on. More: the places of a grid, row by row."""
    m, axes = case["m"], case.get("axes", 1)
    i = torch.arange(m, device="cuda")
    if axes == 1:
        return i + case["start"]
    side = max(1, math.isqrt(m))
    grid = torch.stack((i // side, i % side), 1)
    return grid if axes == 2 else torch.cat((torch.full((m, 1), case["start"] % 1000, device="cuda"), grid), 1)


def _frequencies(case):
    """One per pair, falling with the pair's place on its own axis, stretched for long contexts."""
    f = [torch.arange(n, device="cuda", dtype=torch.float64) / n for n in _axis_pairs(case) if n]
    return 500000.0 ** -torch.cat(f) if f else torch.zeros(0, device="cuda", dtype=torch.float64)


def _heads(g, m, heads, d, dtype):
    """Queries, keys or values as a product leaves them: heads and channels of unlike sizes, a few large channels."""
    x = torch.randn(m, heads, d, generator=g, device="cuda")
    x *= torch.exp(0.4 * torch.randn(heads, d, generator=g, device="cuda"))
    x *= torch.where(torch.rand(heads, d, generator=g, device="cuda") < 0.02, 12.0, 1.0)
    return x.to(dtype)


def prepare(case, seed):
    g = torch.Generator("cuda").manual_seed(seed)
    dtype, m, op = _type(case), case["m"], case["op"]
    s = {"case": dict(case)}
    if op in ("gated", "gated_grad"):
        n = case["n"]
        if op == "gated_grad":
            s["dout"] = torch.randn(m, n, generator=g, device="cuda").to(dtype)
            s["g"], s["u"] = ((1.5 * torch.randn(m, n, generator=g, device="cuda")).to(dtype) for _ in range(2))
            return s
        k = case["k"]
        for name, rows, size in (("a", m, 1.0), ("g", n, k ** -0.5), ("u", n, k ** -0.5)):
            s["codes_" + name], scales = _operand(g, rows, k, size)
            s["scales_" + name] = _pack(scales) if case["packed"] else scales
        for name in ("bias_g", "bias_u"):
            s[name] = 0.5 * torch.randn(n, generator=g, device="cuda") if case["bias"] else None
        return s
    d = case["d"]
    if op in ("head", "head_grad"):
        # the product's output, queries, keys and values side by side; the values are left alone here
        q, k = case["q"], case["k"]
        s["x"] = _heads(g, m, q + 2 * k, d, dtype)[:, :q + k]
        s["weight_q"], s["weight_k"] = (1 + 0.2 * torch.randn(d, generator=g, device="cuda") for _ in range(2))
        s["positions"], s["freq"] = _positions(case, g), _frequencies(case)
        s["amplitude"] = 1.0 if case["start"] < 100000 else 0.1 * math.log(case["start"] / 8192) + 1
        if op == "head_grad":
            s["dy"] = torch.randn(m, q + k, d, generator=g, device="cuda").to(dtype)
        return s
    h = case["h"]
    # pages of 16 rows, taken in no order, a few of them free
    pages = (m + 15) // 16 + 2
    rows = 16 * pages
    order = torch.randperm(pages, generator=g, device="cuda")
    s["slots"] = (16 * order[:, None] + torch.arange(16, device="cuda")).flatten()[:m].contiguous()
    if op == "cache_read":
        codes, scales = _operand(g, rows * h, d, 1.0)
        s["codes"], s["scales"] = codes.view(rows, h, d // 2), scales.view(rows, h, d // 32)
        return s
    codes, scales = _operand(g, 2 * rows * h, d, 1.0)
    s["codes"], s["scales"] = codes.view(2, rows, h, d // 2), scales.view(2, rows, h, d // 32)
    kv = _heads(g, m, 2 * h, d, dtype)
    s["k"], s["v"] = kv[:, :h], kv[:, h:]
    s["weight"] = 1 + 0.2 * torch.randn(d, generator=g, device="cuda") if case["norm"] else None
    s["positions"], s["freq"] = _positions(case, g), _frequencies(case)
    return s


# ---------------------------------------------------------------------------------------------------------
# Plain forms
# ---------------------------------------------------------------------------------------------------------
def _decode(codes, scales, dtype):
    levels = torch.tensor(LEVELS + tuple(-v for v in LEVELS), dtype=dtype, device=codes.device)
    v = torch.stack((levels[(codes & 15).long()], levels[(codes >> 4).long()]), -1)
    v = v.view(*scales.shape, 32)
    return torch.ldexp(v, scales.to(torch.int32)[..., None] - 127).flatten(-2)


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


def _angles(s, dtype):
    """cos and sin of every token's pairs, [m][1][r / 2], times the amplitude; the angles in 64 bits."""
    case = s["case"]
    p = s["positions"].double().view(case["m"], -1)
    axis = torch.tensor([i for i, n in enumerate(_axis_pairs(case)) for _ in range(n)], device=p.device, dtype=torch.long)
    t = p[:, axis] * s["freq"]
    a = s.get("amplitude", 1.0)
    return (torch.cos(t) * a).to(dtype)[:, None], (torch.sin(t) * a).to(dtype)[:, None]


def _rotate(x, cos, sin, inter):
    r = 2 * cos.shape[-1]
    a, b = (x[..., 0:r:2], x[..., 1:r:2]) if inter else (x[..., :r // 2], x[..., r // 2:r])
    a, b = a * cos - b * sin, b * cos + a * sin
    return torch.cat((torch.stack((a, b), -1).flatten(-2) if inter else torch.cat((a, b), -1), x[..., r:]), -1)


def _head_weights(s):
    """[q + k][d], the weight of each head."""
    case = s["case"]
    return torch.cat((s["weight_q"].expand(case["q"], -1), s["weight_k"].expand(case["k"], -1)))


def _plain(s):
    case = s["case"]
    op, dtype = case["op"], _type(case)
    if op == "gated":
        scales = (_unpack(s["scales_" + n]) if case["packed"] else s["scales_" + n] for n in "agu")
        a, wg, wu = (_decode(s["codes_" + n], sc, torch.float32) for n, sc in zip("agu", scales))
        g, u = torch.matmul(a, wg.t()), torch.matmul(a, wu.t())
        if case["bias"]:
            g, u = g + s["bias_g"], u + s["bias_u"]
        out = {"out": (_act(g, case["act"]) * u).to(dtype)}
        if case["pre"]:
            out["g"], out["u"] = g.to(dtype), u.to(dtype)
        return out
    if op == "gated_grad":
        do, g, u = s["dout"].float(), s["g"].float(), s["u"].float()
        dg, du = do * u * _act_grad(g, case["act"]), do * _act(g, case["act"])
        return {"dg": dg.to(dtype), "du": du.to(dtype), "dbias_g": dg.sum(0, dtype=torch.float64).float(),
                "dbias_u": du.sum(0, dtype=torch.float64).float()}
    if op == "cache_read":
        return {"values": _decode(s["codes"][s["slots"]], s["scales"][s["slots"]], torch.float32).to(dtype)}
    if op == "cache_write":
        # in 64 bits: next to a border between two codes the last bit of 32 decides
        k, v = s["k"].double(), s["v"].double()
        if case["norm"]:
            k = k / torch.sqrt((k * k).mean(-1, keepdim=True) + EPS) * s["weight"]
        k = _rotate(k, *_angles(s, torch.float64), case["inter"])
        x = torch.stack((k, v))
        index, e = _indices(x.unflatten(-1, (-1, 32)))
        new = torch.ldexp(torch.tensor(LEVELS, device=x.device)[index.long()], e).flatten(-2)
        values = _decode(s["codes"], s["scales"], torch.float32)
        values[:, s["slots"]] = torch.copysign(new, x.float())
        return {"values": values.to(torch.float8_e5m2)}
    x = s["x"].float()
    w = _head_weights(s)
    cos, sin = _angles(s, torch.float32)
    r = 1 / torch.sqrt((x * x).mean(-1, keepdim=True) + EPS)
    if op == "head":
        return {"y": _rotate(x * r * w, cos, sin, case["inter"]).to(dtype)}
    e = s["dy"].float()
    if case["rot"]:
        # the rotation by the opposite angle
        e = _rotate(e, cos, -sin, case["inter"])
    h = x * r
    ew = e * w
    dx = r * (ew - h * (ew * h).mean(-1, keepdim=True))
    dw = (e * h).double()
    return {"dx": dx.to(dtype), "dweight_q": dw[:, :case["q"]].sum((0, 1)).float(),
            "dweight_k": dw[:, case["q"]:].sum((0, 1)).float()}


def _framework(s):
    import mxfp4_activation_quantizer_amd as kq
    case = s["case"]
    op = case["op"]
    if op == "gated":
        got = kq.mxfp4_gated_linear(s["codes_a"], s["scales_a"], s["codes_g"], s["scales_g"], s["codes_u"],
                                    s["scales_u"], bias_g=s["bias_g"], bias_u=s["bias_u"], act=case["act"],
                                    bf16=case["type"] == "bf16", packed=case["packed"], want_pre=case["pre"])
        return {"out": got[0], "g": got[1], "u": got[2]} if case["pre"] else {"out": got}
    if op == "gated_grad":
        dg, du, dbias_g, dbias_u = kq.mxfp4_gated_linear_backward(s["dout"], s["g"], s["u"], act=case["act"])
        return {"dg": dg, "du": du, "dbias_g": dbias_g, "dbias_u": dbias_u}
    if op == "cache_read":
        return {"values": kq.cache_read_mxfp4(s["slots"], s["codes"], s["scales"], bf16=case["type"] == "bf16")}
    pairs = _axis_pairs(case)
    if op == "cache_write":
        (codes_k, codes_v), (scales_k, scales_v) = s["codes"], s["scales"]
        kq.cache_write_mxfp4(s["slots"], k=s["k"], codes_k=codes_k, scales_k=scales_k, v=s["v"], codes_v=codes_v,
                             scales_v=scales_v, norm=case["norm"], weight=s["weight"], eps=EPS,
                             positions=s["positions"], freq=s["freq"], interleaved=case["inter"])
        # the whole cache as the values that its codes stand for, in a type of 8 bits that holds them all
        d = case["d"]
        values = kq.dequantize_mxfp4_bf16(s["codes"].view(-1, d // 2), s["scales"].view(-1, d // 32))
        return {"values": values.view(*s["codes"].shape[:3], d).to(torch.float8_e5m2)}
    if op == "head":
        return {"y": kq.headnorm_rope(s["x"], s["positions"], s["freq"], weight_q=s["weight_q"],
                                      weight_k=s["weight_k"], q_heads=case["q"], eps=EPS, axis_pairs=pairs,
                                      interleaved=case["inter"], amplitude=s["amplitude"])}
    dx, dweight_q, dweight_k = kq.headnorm_rope_backward(
        s["dy"], s["x"], s["positions"], s["freq"], weight_q=s["weight_q"], weight_k=s["weight_k"],
        q_heads=case["q"], eps=EPS, axis_pairs=pairs, interleaved=case["inter"], amplitude=s["amplitude"])
    return {"dx": dx, "dweight_q": dweight_q, "dweight_k": dweight_k}


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


def _turned(x, s, back):
    """Each pair as a complex number, times exp(i t) of its token (exp(-i t) for the way back) and the amplitude."""
    case = s["case"]
    n = case["rot"] // 2
    if n == 0:
        return x
    p = s["positions"].double().reshape(case["m"], -1)
    t = torch.cat([p[:, i:i + 1].expand(-1, c) for i, c in enumerate(_axis_pairs(case))], 1) * s["freq"]
    turn = torch.polar(torch.full_like(t, s.get("amplitude", 1.0)), -t if back else t)[:, None, :]
    first = 2 * torch.arange(n, device=x.device) if case["inter"] else torch.arange(n, device=x.device)
    second = first + (1 if case["inter"] else n)
    z = torch.complex(x[..., first], x[..., second]) * turn
    y = x.clone()
    y[..., first], y[..., second] = z.real, z.imag
    return y


def exact(case, seed):
    s = prepare(case, seed)
    op, act = case["op"], case.get("act")
    # the codes by their bits: sign, two exponent bits of bias 1, one mantissa bit
    def value(codes, scales):
        c = torch.stack((codes & 15, codes >> 4), -1).flatten(-2).int()
        ex, man = (c >> 1) & 3, (c & 1).double()
        mag = torch.where(ex > 0, (1 + man / 2) * 2.0 ** (ex - 1).double(), man / 2)
        return torch.where(c > 7, -mag, mag) * (2.0 ** (scales.double() - 127)).repeat_interleave(32, -1)

    if op == "cache_write":
        # the codes are steps of their inputs: next to a border no number of bits makes one side the right one
        return None
    if op == "cache_read":
        return {"values": value(s["codes"], s["scales"])[s["slots"]]}
    if op == "gated":
        a, wg, wu = (value(s["codes_" + n], _unpack(s["scales_" + n]) if case["packed"] else s["scales_" + n])
                     for n in "agu")
        g, u = a @ wg.T, a @ wu.T
        if case["bias"]:
            g += s["bias_g"].double()
            u += s["bias_u"].double()
        out = {"out": _exact_act(g, act)[0] * u}
        return {**out, "g": g, "u": u} if case["pre"] else out
    if op == "gated_grad":
        f, slope = _exact_act(s["g"].double(), act)
        do = s["dout"].double()
        dg, du = do * slope * s["u"].double(), do * f
        return {"dg": dg, "du": du, "dbias_g": dg.sum(0), "dbias_u": du.sum(0)}
    x, q = s["x"].double(), case["q"]
    rms = (torch.linalg.vector_norm(x, dim=-1, keepdim=True) ** 2 / case["d"] + EPS) ** 0.5
    weight = torch.empty_like(x)
    weight[:, :q], weight[:, q:] = s["weight_q"].double(), s["weight_k"].double()
    if op == "head":
        return {"y": _turned(x / rms * weight, s, False)}
    e = _turned(s["dy"].double(), s, True)
    h = x / rms
    b = torch.linalg.vecdot(e * weight, h)[..., None] / case["d"]
    dw = (e * h).sum(0)
    return {"dx": (e * weight - h * b) / rms, "dweight_q": dw[:q].sum(0), "dweight_k": dw[q:].sum(0)}
