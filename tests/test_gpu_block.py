"""GPU: a transformer block out of the framework's operators, as a program runs it -- norm into the quantizer, the product
of queries, keys and values, their norm and rotation, the MXFP4 cache with an attention over what it reads back, the gated
feed-forward product -- for a prompt, then token by token in a captured graph, on another stream, and the way back. Each
step is held against 64 bits at what the step before it gave."""
import pytest

from tests import gated_ref, heads_ref
from tests import layer_ref as ref

pytestmark = pytest.mark.gpu

EPS = 1e-5


@pytest.fixture(scope="module")
def torch():
    import torch
    assert torch.cuda.is_available(), "GPU tests need a HIP device"
    return torch


@pytest.fixture(scope="module")
def kq():
    import mxfp4_activation_quantizer_amd as kq
    kq.lib()
    return kq


class Block:
    """y = x + Wo attention(heads(Wqkv Q(LN x))), then y + Wd Q(act(Wg Q(LN y)) * Wu Q(LN y))."""

    def __init__(self, torch, kq, width, q, kv, d, rot, inner, act, inter, capacity, dtype):
        self.torch, self.kq = torch, kq
        self.width, self.q, self.kv, self.d, self.inner, self.act, self.inter = width, q, kv, d, inner, act, inter
        self.dtype, self.bf16 = dtype, dtype is torch.bfloat16
        g = torch.Generator("cuda").manual_seed(width + inner)

        def weight(n, k):
            w = torch.randn(n, k, generator=g, device="cuda") * k ** -0.5
            codes, scales = kq.quantize_mxfp4_f32(w)
            return codes, scales, kq.pack_mxfp4_scales(scales) if k % 256 == 0 else scales, k % 256 == 0

        self.w_qkv, self.w_o = weight((q + 2 * kv) * d, width), weight(width, q * d)
        self.w_g, self.w_u, self.w_d = weight(inner, width), weight(inner, width), weight(width, inner)
        self.norm = [1 + 0.1 * torch.randn(width, generator=g, device="cuda") for _ in range(2)]
        self.norm_q, self.norm_k = (1 + 0.1 * torch.randn(d, generator=g, device="cuda") for _ in range(2))
        self.bias_g, self.bias_u = (0.1 * torch.randn(inner, generator=g, device="cuda") for _ in range(2))
        self.freq = torch.from_numpy(kq.rope_frequencies(rot)).cuda()
        self.codes = torch.zeros(2, capacity, kv, d // 2, dtype=torch.uint8, device="cuda")
        self.scales = torch.zeros(2, capacity, kv, d // 32, dtype=torch.uint8, device="cuda")

    def quantize(self, x, packed):
        codes, scales = self.kq.quantize_mxfp4(x) if self.bf16 else self.kq.quantize_mxfp4_f32(x)
        return codes, self.kq.pack_mxfp4_scales(scales) if packed else scales

    def linear(self, codes, scales, w, residual=None):
        return self.kq.mxfp4_linear(codes, scales, w[0], w[2], residual=residual, bf16=self.bf16, packed=w[3])

    def rope(self, positions):
        return dict(positions=positions, freq=self.freq, interleaved=self.inter)

    def attention(self, queries, keys, values, seen):
        """Plain: queries [m][q][d] over the cache's rows; seen: bool [m][rows]. Sums over rows without a library product,
        so that a row's result does not depend on the others."""
        torch = self.torch
        k, v = (t.float().repeat_interleave(self.q // self.kv, 1) for t in (keys, values))
        s = (queries.float()[:, None] * k[None]).sum(-1) * self.d ** -0.5
        p = torch.softmax(s.masked_fill(~seen[:, :, None], -torch.inf), 1)
        return (p[..., None] * v[None]).sum(1).to(self.dtype).flatten(1)

    def forward(self, x, positions, slots, pages, seen):
        """x [m][width] of tokens at `positions`, written to `slots`, each seeing `seen` of the slots `pages`."""
        kq, kept = self.kq, {}
        m, qd, kd = x.shape[0], self.q * self.d, self.kv * self.d
        kept["a1"] = kq.layernorm_quantize_mxfp4(x, self.norm[0], None, eps=EPS, packed=self.w_qkv[3])
        qkv = kept["qkv"] = self.linear(*kept["a1"], self.w_qkv)
        heads = qkv.view(m, -1, self.d)
        kept["queries"] = kq.headnorm_rope(heads[:, :self.q], weight_q=self.norm_q, eps=EPS, **self.rope(positions))
        kq.cache_write_mxfp4(slots, k=heads[:, self.q:self.q + self.kv], codes_k=self.codes[0], scales_k=self.scales[0],
                             v=heads[:, self.q + self.kv:], codes_v=self.codes[1], scales_v=self.scales[1], norm=True,
                             weight=self.norm_k, eps=EPS, **self.rope(positions))
        kept["keys"], kept["values"] = (kq.cache_read_mxfp4(pages, self.codes[i], self.scales[i], bf16=self.bf16)
                                        for i in range(2))
        mixed = kept["mixed"] = self.attention(kept["queries"], kept["keys"], kept["values"], seen)
        y = kept["y"] = self.linear(*self.quantize(mixed, self.w_o[3]), self.w_o, x)
        kept["a2"] = kq.layernorm_quantize_mxfp4(y, self.norm[1], None, eps=EPS, packed=self.w_g[3])
        kept["gated"], kept["g"], kept["u"] = kq.mxfp4_gated_linear(
            *kept["a2"], self.w_g[0], self.w_g[2], self.w_u[0], self.w_u[2], self.bias_g, self.bias_u, act=self.act,
            bf16=self.bf16, packed=self.w_g[3], want_pre=True)
        kept["out"] = self.linear(*self.quantize(kept["gated"], self.w_d[3]), self.w_d, y)
        return kept

    def unpacked(self, a, w, m):
        return a[0], ref.unpack_scales(a[1], m, 2 * a[0].shape[1]) if w[3] else a[1]


def prompt(torch, block, m, order, pages):
    g = torch.Generator("cuda").manual_seed(m)
    x = torch.randn(m, block.width, generator=g, device="cuda").to(block.dtype)
    positions = torch.arange(m, device="cuda")
    slots = order[:m].contiguous()
    seen = positions[:, None] >= torch.arange(pages.numel(), device="cuda")
    return x, positions, slots, pages, seen


SHAPES = [  # width, query and key heads, channels, rotated, inner width, tokens
    (544, 3, 1, 32, 32, 864, 19, "gelu", False),
    (768, 8, 2, 64, 32, 1280, 40, "silu", True),
    (256, 4, 4, 96, 96, 512, 65, "gelu_tanh", False),
    (1024, 8, 4, 128, 128, 2048, 1, "silu", False),
]


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
@pytest.mark.parametrize("width,q,kv,d,rot,inner,m,act,inter", SHAPES)
def test_prompt_step_by_step(torch, kq, width, q, kv, d, rot, inner, m, act, inter, dtype):
    block = Block(torch, kq, width, q, kv, d, rot, inner, act, inter, m + 7, getattr(torch, dtype))
    order = torch.randperm(m + 7, generator=torch.Generator().manual_seed(m)).cuda()
    args = prompt(torch, block, m, order, order[:m].contiguous())
    positions, slots = args[1], args[2]
    kept = block.forward(*args)
    # the product, at the codes that the norm wrote
    want, _, tol, _ = ref.linear(*block.unpacked(kept["a1"], block.w_qkv, m), *block.w_qkv[:2], None, "none", None)
    ref.assert_near(kept["qkv"], want, tol, "qkv")
    heads = kept["qkv"].view(m, -1, d)
    rope = dict(positions=positions, freq=block.freq, inter=inter)
    want, tol = heads_ref.forward(heads[:, :q], block.norm_q, None, q, EPS, rope)
    ref.assert_near(kept["queries"], want, tol, "queries")
    want, tol = heads_ref.forward(heads[:, q:q + kv], block.norm_k, None, kv, EPS, rope)
    heads_ref.assert_codes_near(block.codes[0][slots], block.scales[0][slots], want, tol, "keys")
    values = heads[:, q + kv:].double()
    heads_ref.assert_codes_near(block.codes[1][slots], block.scales[1][slots], values, 0 * values, "values")
    rest = torch.ones(m + 7, dtype=torch.bool, device="cuda")
    rest[slots] = False
    assert not block.codes[:, rest].any() and not block.scales[:, rest].any(), "slots of no token"
    for i, name in enumerate(("keys", "values")):
        back = ref.decode(block.codes[i][slots].flatten(0, 1), block.scales[i][slots].flatten(0, 1)).view(m, kv, d)
        assert torch.equal(kept[name].double(), back), name  # four bits and a power of two: no rounding
    mixed = block.quantize(kept["mixed"], block.w_o[3])
    want, _, tol, _ = ref.linear(*block.unpacked(mixed, block.w_o, m), *block.w_o[:2], None, "none", args[0])
    ref.assert_near(kept["y"], want, tol, "y")
    a2 = block.unpacked(kept["a2"], block.w_g, m)
    o, g, u, o_tol, g_tol, u_tol = gated_ref.forward(*a2, *block.w_g[:2], *block.w_u[:2], block.bias_g, block.bias_u, act,
                                                     block.dtype)
    for name, want, tol in (("gated", o, o_tol), ("g", g, g_tol), ("u", u, u_tol)):
        ref.assert_near(kept[name], want, tol, name)
    down = block.unpacked(block.quantize(kept["gated"], block.w_d[3]), block.w_d, m)
    want, _, tol, _ = ref.linear(*down, *block.w_d[:2], None, "none", kept["y"])
    ref.assert_near(kept["out"], want, tol, "out")


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
def test_tokens_in_a_graph_and_on_another_stream(torch, kq, dtype):
    """One captured graph serves every later token, its position and slot written into the graph's own tensors; between its
    replays the eager block works on a cache of its own, on another stream. Each replay gives the eager results bit by bit."""
    shape, capacity, m = (768, 8, 2, 64, 32, 1280), 64, 21
    eager, graphed = (Block(torch, kq, *shape, "silu", False, capacity, getattr(torch, dtype)) for _ in range(2))
    order = torch.randperm(capacity, generator=torch.Generator().manual_seed(5)).cuda()
    first = prompt(torch, eager, m, order, order)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        before = eager.forward(*first)
    after = graphed.forward(*first)
    torch.cuda.synchronize()
    for name in ("out", "queries", "keys", "values", "gated"):
        assert torch.equal(before[name], after[name]), name
    tokens = torch.randn(9, 1, 768, generator=torch.Generator("cuda").manual_seed(9), device="cuda").to(eager.dtype)
    rows = torch.arange(capacity, device="cuda")
    x, position, slot = tokens[0].clone(), torch.full((1,), m, device="cuda"), order[m:m + 1].clone()

    def token(block, x, position, slot):
        return block.forward(x, position, slot, order, position[:, None] >= rows)

    kept = (graphed.codes.clone(), graphed.scales.clone())
    warm = torch.cuda.Stream()
    warm.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(warm):
        token(graphed, x, position, slot)
    torch.cuda.current_stream().wait_stream(warm)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = token(graphed, x, position, slot)
    graphed.codes.copy_(kept[0])
    graphed.scales.copy_(kept[1])
    for i in range(tokens.shape[0]):
        x.copy_(tokens[i])
        position.fill_(m + i)
        slot.copy_(order[m + i:m + i + 1])
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            want = token(eager, tokens[i], torch.full((1,), m + i, device="cuda"), order[m + i:m + i + 1].clone())
        graph.replay()
        torch.cuda.synchronize()
        for name in ("out", "queries", "keys", "values", "gated", "g", "u"):
            assert torch.equal(got[name], want[name]), (i, name)
        assert torch.equal(eager.codes, graphed.codes) and torch.equal(eager.scales, graphed.scales), i


@pytest.mark.parametrize("width,q,kv,d,rot,inner,m,act,inter", SHAPES)
def test_the_way_back(torch, kq, width, q, kv, d, rot, inner, m, act, inter):
    """Straight through the quantizers, fp32: from the block's output to the input of the gated products, and from queries,
    keys and values to the input of theirs, against the formulas in 64 bits."""
    block = Block(torch, kq, width, q, kv, d, rot, inner, act, inter, m, torch.float32)
    order = torch.arange(m, device="cuda")
    args = prompt(torch, block, m, order, order)
    kept = block.forward(*args)
    gen = torch.Generator("cuda").manual_seed(inner)
    dout = torch.randn(m, width, generator=gen, device="cuda")
    w_d, w_g, w_u, w_qkv = (ref.decode(*w[:2]) for w in (block.w_d, block.w_g, block.w_u, block.w_qkv))

    def product(n):  # a product of n terms in fp32, of the sum of their absolute values
        return (n + 2) * 2.0 ** -22

    dh = kq.gemm_f32(dout, w_d.float())
    dg, du, dbias_g, dbias_u = kq.mxfp4_gated_linear_backward(dh, kept["g"], kept["u"], act=act)
    da = kq.gemm_f32(dg, w_g.float()) + kq.gemm_f32(du, w_u.float())
    dh64 = dout.double() @ w_d
    off = product(width) * (dout.double().abs() @ w_d.abs())
    (dg64, du64, bg64, bu64), (dg_tol, du_tol, bg_tol, bu_tol) = gated_ref.backward(dh64, kept["g"], kept["u"], act)
    # linear in dh: what dh is off by, times the factors that it meets (their own error in second order: 1.01)
    act64, slope, _, _ = gated_ref.value(kept["g"].double(), act, torch.float32)
    dg_tol = 1.01 * (dg_tol + off * (kept["u"].double() * slope).abs()) + ref.half_step(dg.dtype, dg64)
    du_tol = 1.01 * (du_tol + off * act64.abs()) + ref.half_step(du.dtype, du64)
    ref.assert_near(dg, dg64, dg_tol, "dg")
    ref.assert_near(du, du64, du_tol, "du")
    ref.assert_near(dbias_g, bg64, 1.01 * bg_tol + dg_tol.sum(0), "dbias_g")
    ref.assert_near(dbias_u, bu64, 1.01 * bu_tol + du_tol.sum(0), "dbias_u")
    da64 = dg64 @ w_g + du64 @ w_u
    size = dg64.abs() @ w_g.abs() + du64.abs() @ w_u.abs()
    ref.assert_near(da, da64, 1.01 * (dg_tol @ w_g.abs() + du_tol @ w_u.abs() + product(inner) * size) + ref.U * da64.abs(),
                    "the gated products' input")

    # queries and keys in one call, into their part of the product's gradient; values pass
    heads = kept["qkv"].view(m, -1, d)
    dheads = torch.randn(m, q + 2 * kv, d, generator=gen, device="cuda")
    dqkv = torch.empty_like(kept["qkv"])
    into = dqkv.view(m, -1, d)
    into[:, q + kv:] = dheads[:, q + kv:]
    _, dwq, dwk = kq.headnorm_rope_backward(dheads[:, :q + kv], heads[:, :q + kv], args[1], block.freq, weight_q=block.norm_q,
                                            weight_k=block.norm_k, q_heads=q, eps=EPS, interleaved=inter,
                                            dx=into[:, :q + kv])
    rope = dict(positions=args[1], freq=block.freq, inter=inter)
    (dx64, wq64, wk64), (dx_tol, wq_tol, wk_tol) = heads_ref.backward(dheads[:, :q + kv], heads[:, :q + kv], block.norm_q,
                                                                     block.norm_k, q, EPS, rope)
    dx_tol = dx_tol + ref.half_step(dqkv.dtype, dx64)
    ref.assert_near(into[:, :q + kv], dx64, dx_tol, "dqk")
    ref.assert_near(dwq, wq64, wq_tol, "dweight_q")
    ref.assert_near(dwk, wk64, wk_tol, "dweight_k")
    assert torch.equal(into[:, q + kv:], dheads[:, q + kv:])
    d64 = torch.cat((dx64, dheads[:, q + kv:].double()), 1).flatten(1)
    d_tol = torch.cat((dx_tol, 0 * dheads[:, q + kv:].double()), 1).flatten(1)
    dx = kq.gemm_f32(dqkv, w_qkv.float())
    ref.assert_near(dx, d64 @ w_qkv, 1.01 * (d_tol @ w_qkv.abs() + product(dqkv.shape[1]) * (d64.abs() @ w_qkv.abs())),
                    "the product's input")
