"""GPU: the norm of query and key heads with the rotation in the same pass (kq_headnorm_rope), its gradients, and
the MXFP4 cache of keys and values, against 64-bit forms (tests/heads_ref.py)."""
import math

import pytest

from tests import heads_ref as ref
from tests import layer_ref

pytestmark = pytest.mark.gpu

EPS = 1e-6


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


def make_heads(torch, g, m, heads, d, dtype):
    x = torch.randn(m, heads, d, generator=g, device="cuda")
    x *= torch.exp(0.5 * torch.randn(heads, d, generator=g, device="cuda"))
    return x.to(dtype)


def make_rope(torch, g, m, rot, inter, axes=1, amplitude=1.0, far=5000):
    n = rot // 2
    pairs = tuple(n // axes + (1 if i < n % axes else 0) for i in range(axes))
    freq = torch.cat([10000.0 ** -(torch.arange(c, dtype=torch.float64) / max(c, 1)) for c in pairs]).cuda()
    shape = (m,) if axes == 1 else (m, axes)
    positions = torch.randint(-far // 8, far, shape, generator=g, device="cuda")
    return {"positions": positions, "freq": freq, "inter": inter, "axis_pairs": pairs, "amplitude": amplitude}


def call_args(rope):
    return dict(positions=rope["positions"], freq=rope["freq"], interleaved=rope["inter"],
                axis_pairs=rope["axis_pairs"], amplitude=rope["amplitude"])


# (m, heads, q heads, d, rot): every width of a piece, every group of lanes, parts of heads that are rotated, odd
# numbers of pieces, heads that do not fill a wave, blocks of tokens and a last partial one
FORMS = [(1, 1, 1, 128, 128), (1, 40, 32, 128, 128), (3, 5, 2, 32, 32), (7, 9, 9, 64, 32), (5, 6, 0, 128, 64),
         (2, 3, 1, 256, 256), (9, 4, 3, 512, 512), (2, 3, 2, 1024, 1024), (3, 2, 1, 1024, 0), (4, 5, 3, 88, 48),
         (6, 7, 4, 72, 72), (3, 2, 1, 40, 40), (2, 2, 1, 120, 120), (3, 3, 2, 252, 252), (2, 3, 1, 516, 504),
         (2, 2, 1, 1020, 1020), (33, 3, 2, 20, 8), (2, 5, 3, 1, 0), (3, 2, 1, 2, 2), (4, 3, 2, 3, 2), (5, 2, 1, 65, 64),
         (2, 3, 2, 130, 130), (2, 2, 1, 257, 198), (1, 2, 1, 1023, 1022), (2, 2, 1, 510, 6), (300, 3, 2, 96, 96),
         (1500, 2, 1, 48, 16), (700, 12, 8, 64, 64), (1100, 40, 32, 128, 128), (1300, 16, 16, 72, 72)]


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("m,heads,q,d,rot", FORMS)
def test_forward_and_gradients(torch, kq, m, heads, q, d, rot, inter, dtype):
    dtype = getattr(torch, dtype)
    g = torch.Generator("cuda").manual_seed(1000 * d + rot + m)
    x = make_heads(torch, g, m, heads, d, dtype)
    wq, wk = (1 + 0.2 * torch.randn(d, generator=g, device="cuda") for _ in range(2))
    rope = make_rope(torch, g, m, rot, inter)
    y = kq.headnorm_rope(x, weight_q=wq, weight_k=wk, q_heads=q, eps=EPS, **call_args(rope))
    want, tol = ref.forward(x, wq, wk, q, EPS, rope)
    layer_ref.assert_near(y, want, tol, "y")
    dy = torch.randn(m, heads, d, generator=g, device="cuda").to(dtype)
    got = kq.headnorm_rope_backward(dy, x, weight_q=wq, weight_k=wk, q_heads=q, eps=EPS, **call_args(rope))
    want, tol = ref.backward(dy, x, wq, wk, q, EPS, rope)
    for name, a, b, t in zip(("dx", "dweight_q", "dweight_k"), got, want, tol):
        layer_ref.assert_near(a, b, t, name)
    again = kq.headnorm_rope_backward(dy, x, weight_q=wq, weight_k=wk, q_heads=q, eps=EPS, **call_args(rope))
    assert all(torch.equal(a, b) for a, b in zip(got, again))


@pytest.mark.parametrize("d,rot,axes", [(128, 128, 3), (72, 72, 2), (64, 32, 4), (66, 66, 3), (16, 2, 2)])
@pytest.mark.parametrize("inter", [False, True])
def test_axes_amplitude_and_far_positions(torch, kq, d, rot, axes, inter):
    g = torch.Generator("cuda").manual_seed(d + axes)
    m, heads = 37, 3
    x = make_heads(torch, g, m, heads, d, torch.float32)
    rope = make_rope(torch, g, m, rot, inter, axes, amplitude=1.25, far=1 << 40)
    want, tol = ref.forward(x, None, None, heads, EPS, rope)
    layer_ref.assert_near(kq.headnorm_rope(x, eps=EPS, **call_args(rope)), want, tol, "y")
    # the rotation alone, and its way back
    want, tol = ref.forward(x, None, None, heads, EPS, rope, norm=False)
    layer_ref.assert_near(kq.headnorm_rope(x, norm=False, **call_args(rope)), want, tol, "rotation alone")
    want, tol = ref.backward(x, None, None, None, heads, EPS, rope, norm=False)
    dx, dq, dk = kq.headnorm_rope_backward(x, norm=False, **call_args(rope))
    layer_ref.assert_near(dx, want[0], tol[0], "rotation back")
    assert dq is None and dk is None


def test_norm_alone(torch, kq):
    g = torch.Generator("cuda").manual_seed(3)
    x = make_heads(torch, g, 11, 4, 128, torch.bfloat16)
    want, tol = ref.forward(x, None, None, 4, EPS, None)
    layer_ref.assert_near(kq.headnorm_rope(x, eps=EPS), want, tol, "y")


def strided(torch, t, token_gap, head_gap, head_major=False, shift=0):
    """t's values in a larger buffer of NaNs: tokens and heads apart by more than they need."""
    m, heads, d = t.shape
    a, b = (heads, m) if head_major else (m, heads)
    inner, outer = d + head_gap, (d + head_gap) * b + token_gap
    base = torch.full((shift + a * outer + 64,), math.nan, dtype=t.dtype, device="cuda")
    strides = (inner, outer, 1) if head_major else (outer, inner, 1)
    view = base.as_strided((m, heads, d), strides, shift)
    view.copy_(t)
    return base, view


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
@pytest.mark.parametrize("shift,token_gap,head_gap,head_major", [
    (0, 64, 0, False), (8, 16, 8, True), (4, 4, 4, False), (1, 3, 5, False), (0, 8, 0, True), (2, 0, 2, True)])
@pytest.mark.parametrize("d,rot,inter", [(64, 64, False), (96, 32, True), (45, 44, False)])
def test_strides(torch, kq, dtype, d, rot, inter, shift, token_gap, head_gap, head_major):
    """Addresses and strides of every kind give the contiguous call's bits; nothing else is read or written."""
    dtype = getattr(torch, dtype)
    g = torch.Generator("cuda").manual_seed(d + shift)
    m, heads, q = 13, 5, 3
    x = make_heads(torch, g, m, heads, d, dtype)
    dy = torch.randn(m, heads, d, generator=g, device="cuda").to(dtype)
    wq, wk = (1 + 0.2 * torch.randn(d, generator=g, device="cuda") for _ in range(2))
    rope = make_rope(torch, g, m, rot, inter)
    kw = dict(weight_q=wq, weight_k=wk, q_heads=q, eps=EPS, **call_args(rope))
    want, tol = ref.forward(x, wq, wk, q, EPS, rope)
    _, xs = strided(torch, x, token_gap, head_gap, head_major, shift)
    base, out = strided(torch, x, token_gap, head_gap, head_major, shift)
    base.fill_(math.nan)
    before = base.clone()
    assert kq.headnorm_rope(xs, out=out, **kw) is out
    layer_ref.assert_near(out, want, tol, "y")
    out.fill_(math.nan)
    assert torch.equal(base.view(torch.uint8), before.view(torch.uint8)), "written outside the heads"
    _, dys = strided(torch, dy, token_gap, head_gap, head_major, shift)
    dx, dq, dk = kq.headnorm_rope_backward(dys, xs, dx=out, **kw)
    want, tol = ref.backward(dy, x, wq, wk, q, EPS, rope)
    for name, a, b, t in zip(("dx", "dweight_q", "dweight_k"), (dx, dq, dk), want, tol):
        layer_ref.assert_near(a, b, t, name)
    out.fill_(math.nan)
    assert torch.equal(base.view(torch.uint8), before.view(torch.uint8)), "written outside the heads"


def test_in_place_and_broadcast(torch, kq):
    g = torch.Generator("cuda").manual_seed(9)
    x = make_heads(torch, g, 200, 6, 128, torch.bfloat16)
    rope = make_rope(torch, g, 200, 128, False)
    want = kq.headnorm_rope(x, eps=EPS, **call_args(rope))
    y = x.clone()
    assert kq.headnorm_rope(y, out=y, eps=EPS, **call_args(rope)) is y
    assert torch.equal(y, want)
    # one gradient for all heads and tokens
    dy = torch.randn(1, 1, 128, generator=g, device="cuda").to(torch.bfloat16)
    a = kq.headnorm_rope_backward(dy.expand(200, 6, 128), x, eps=EPS, **call_args(rope))
    b = kq.headnorm_rope_backward(dy.expand(200, 6, 128).contiguous(), x, eps=EPS, **call_args(rope))
    assert all(torch.equal(i, j) for i, j in zip(a, b))
    # the gradient in its own place
    own = dy.expand(200, 6, 128).contiguous()
    c = kq.headnorm_rope_backward(own, x, dx=own, eps=EPS, **call_args(rope))
    assert all(torch.equal(i, j) for i, j in zip(a, c))


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
def test_a_bad_head_stays_alone(torch, kq, bad):
    g = torch.Generator("cuda").manual_seed(10)
    for d in (128, 72, 33):
        x = make_heads(torch, g, 20, 7, d, torch.float32)
        rope = make_rope(torch, g, 20, d // 2 * 2, False)
        clean = kq.headnorm_rope(x, eps=EPS, **call_args(rope))
        x[11, 3, d // 2] = bad
        y = kq.headnorm_rope(x, eps=EPS, **call_args(rope))
        assert bool(torch.isnan(y[11, 3]).any())
        y[11, 3] = clean[11, 3]
        assert torch.equal(y, clean)


def test_zero_heads_and_small_values(torch, kq):
    x = torch.zeros(3, 2, 64, device="cuda")
    x[1] = 1e-18
    y = kq.headnorm_rope(x, eps=EPS)
    want, tol = ref.forward(x, None, None, 2, EPS, None)
    assert bool((y[0] == 0).all())
    layer_ref.assert_near(y, want, tol, "y")
    got = kq.headnorm_rope_backward(torch.ones_like(x), x, eps=EPS)
    want, tol = ref.backward(torch.ones_like(x), x, None, None, 2, EPS, None)
    for a, b, t in zip(got, want, tol):
        layer_ref.assert_near(a, b, t)


def test_nothing_to_do(torch, kq):
    x = torch.empty(0, 4, 64, device="cuda")
    assert kq.headnorm_rope(x).shape == (0, 4, 64)
    dx, dq, dk = kq.headnorm_rope_backward(x, x, dweight_q=torch.full((64,), 7.0, device="cuda"))
    assert dx.shape == x.shape and bool((dq == 0).all()) and bool((dk == 0).all())
    x = torch.empty(5, 0, 64, device="cuda")
    _, dq, dk = kq.headnorm_rope_backward(x, x)
    assert bool((dq == 0).all()) and bool((dk == 0).all())
    assert kq.headnorm_rope(torch.empty(5, 2, 0, device="cuda")).numel() == 0
    # heads of one kind only: the other weight's gradient is zeros
    g = torch.Generator("cuda").manual_seed(1)
    x = make_heads(torch, g, 9, 3, 32, torch.float32)
    for q, zero in ((3, 2), (0, 1)):
        got = kq.headnorm_rope_backward(x, x, q_heads=q)
        assert bool((got[zero] == 0).all()) and bool((got[3 - zero] != 0).any())


def test_each_gradient_alone(torch, kq):
    """Through the C entry point: a NULL dweight is left out, the other's bits stay."""
    g = torch.Generator("cuda").manual_seed(4)
    x = make_heads(torch, g, 50, 4, 64, torch.float32)
    dy = torch.randn_like(x)
    dx, dq, dk = kq.headnorm_rope_backward(dy, x, q_heads=3, eps=EPS)
    ws = torch.empty(1 << 20, dtype=torch.uint8, device="cuda")
    for want_q in (True, False):
        one, out = torch.empty(64, device="cuda"), torch.empty_like(x)
        kq._check("kq_headnorm_rope_backward", kq.lib().kq_headnorm_rope_backward(
            dy.data_ptr(), 256, 64, x.data_ptr(), 256, 64, 0, 50, 4, 64, 1, None, None, 3, EPS, None, out.data_ptr(),
            256, 64, one.data_ptr() if want_q else None, None if want_q else one.data_ptr(), ws.data_ptr(), ws.numel(),
            torch.cuda.current_stream().cuda_stream))
        assert torch.equal(one, dq if want_q else dk) and torch.equal(out, dx)


def test_gradient_against_differences(torch, kq):
    """The kernel's gradient along a direction, and a central difference of the 64-bit form: its error is the third
    derivative's, e^2 of the loss's size, and 2^-52 of it over e."""
    g = torch.Generator("cuda").manual_seed(5)
    m, heads, q, d = 6, 5, 3, 48
    x = make_heads(torch, g, m, heads, d, torch.float32)
    dy = torch.randn(m, heads, d, generator=g, device="cuda")
    wq, wk = (1 + 0.2 * torch.randn(d, generator=g, device="cuda") for _ in range(2))
    rope = make_rope(torch, g, m, 32, True, amplitude=1.1)
    got = kq.headnorm_rope_backward(dy, x, weight_q=wq, weight_k=wk, q_heads=q, eps=EPS, **call_args(rope))
    _, tol = ref.backward(dy, x, wq, wk, q, EPS, rope)

    def loss(x, wq, wk):
        return (ref.forward(x, wq, wk, q, EPS, rope)[0] * dy.double()).sum()

    e = 1e-5
    at = [x.double(), wq.double(), wk.double()]
    for i in range(3):
        v = torch.randn(at[i].shape, generator=g, device="cuda", dtype=torch.float64)
        up, down = ([t + s * e * v if j == i else t for j, t in enumerate(at)] for s in (1, -1))
        diff = (loss(*up) - loss(*down)) / (2 * e)
        # a direction's third derivative is at most 100 times sum |dy| |v|^3 here (heads of size 1 and weights near 1)
        slack = (tol[i] * v.abs()).sum() + layer_ref.half_step(got[i].dtype, got[i].double().abs()).mul(v.abs()).sum() \
            + 100 * e * e * (dy.abs().double().sum() * 30) + 2.0 ** -50 * dy.abs().double().sum() * 4 / e
        assert abs(float(diff - (got[i].double() * v).sum())) <= float(slack)


def test_other_streams_and_graphs(torch, kq):
    g = torch.Generator("cuda").manual_seed(6)
    x = make_heads(torch, g, 300, 6, 128, torch.bfloat16)
    dy = torch.randn(300, 6, 128, generator=g, device="cuda").to(torch.bfloat16)
    rope = make_rope(torch, g, 300, 128, False)
    kw = dict(q_heads=4, eps=EPS, **call_args(rope))
    want = (kq.headnorm_rope(x, **kw), *kq.headnorm_rope_backward(dy, x, **kw))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [None, None]
    for _ in range(4):
        for i, s in enumerate(streams):
            got[i] = (kq.headnorm_rope(x, stream=s, **kw), *kq.headnorm_rope_backward(dy, x, stream=s, **kw))
    torch.cuda.synchronize()
    for o in got:
        assert all(torch.equal(a, b) for a, b in zip(o, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = (kq.headnorm_rope(x, **kw), *kq.headnorm_rope_backward(dy, x, **kw))
    for step in range(3):
        x.copy_(make_heads(torch, g, 300, 6, 128, torch.bfloat16))
        rope["positions"].add_(step)
        graph.replay()
        torch.cuda.synchronize()
        want = (kq.headnorm_rope(x, **kw), *kq.headnorm_rope_backward(dy, x, **kw))
        assert all(torch.equal(a, b) for a, b in zip(out, want)), step


@pytest.mark.parametrize("m", [5, 8])
def test_most_heads(torch, kq, m):
    """As many heads as there can be, one wave each, several tokens to a workgroup: their passes are divided into tokens."""
    g = torch.Generator("cuda").manual_seed(m)
    heads, d = 65536, 34
    x, dy = (torch.randn(m, heads, d, generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    kw = dict(eps=EPS, **call_args(make_rope(torch, g, m, 34, False)))
    y, (dx, dq, dk) = kq.headnorm_rope(x, **kw), kq.headnorm_rope_backward(dy, x, q_heads=heads - 1, **kw)
    parts = []
    for i in range(0, heads, 8192):
        a, b = x[:, i:i + 8192], dy[:, i:i + 8192]
        da, q, k = kq.headnorm_rope_backward(b, a, q_heads=min(8192, heads - 1 - i), **kw)
        assert torch.equal(y[:, i:i + 8192], kq.headnorm_rope(a, **kw)), i
        assert torch.equal(dx[:, i:i + 8192], da), i
        parts.append((q.double(), k.double()))
    # the same terms in another order: chains of at most m heads / 8 of them and the joins, in both
    e, h = dy.float().abs(), x.float().abs()
    size = ((e + e.roll(17, -1)) * h * h.square().mean(-1, keepdim=True).rsqrt()).sum((0, 1), dtype=torch.float64)
    for got, want in zip((dq, dk), zip(*parts)):
        assert bool(((got - sum(want)).abs() <= 2 * (m * heads / 8 + 64) * 2.0 ** -24 * size).all())
    alone = kq.headnorm_rope_backward(dy[:, -1:], x[:, -1:], q_heads=0, **kw)[2]
    assert bool(((dk - alone).abs() <= 64 * 2.0 ** -24 * (dy[:, -1].abs().float() * 8).sum(0).max()).all())


@pytest.mark.parametrize("d,rot,inter", [(128, 128, False), (20, 8, True), (30, 30, False)])
@pytest.mark.parametrize("heads", [8, 1])
def test_strides_past_a_pass(torch, kq, d, rot, inter, heads):
    """Heads (or tokens) so far from each other that the lanes of a wave, on several at once, would not reach the last of
    them with 31 bits."""
    g = torch.Generator("cuda").manual_seed(d)
    n, gap = 8, -(-(1 << 30) // (2 if d == 30 else 6))
    gap += -gap % 128
    m = 3 if heads == 8 else n

    def far():
        flat = torch.empty((n - 1) * gap + 3 * d + 128, dtype=torch.bfloat16, device="cuda")
        return flat.as_strided((m, heads, d), (d, gap, 1) if heads == 8 else (gap, d, 1))

    x, dy, out, dx = (far() for _ in range(4))
    x.copy_(make_heads(torch, g, m, heads, d, torch.bfloat16))
    dy.copy_(torch.randn(m, heads, d, generator=g, device="cuda"))
    rope = make_rope(torch, g, m, rot, inter)
    kw = dict(eps=EPS, **call_args(rope))
    kq.headnorm_rope(x, out=out, **kw)
    want, tol = ref.forward(x, None, None, heads, EPS, rope)
    layer_ref.assert_near(out, want, tol, "y")
    _, dq, _ = kq.headnorm_rope_backward(dy, x, dx=dx, **kw)
    want, tol = ref.backward(dy, x, None, None, heads, EPS, rope)
    layer_ref.assert_near(dx, want[0], tol[0], "dx")
    layer_ref.assert_near(dq, want[1], tol[1], "dweight")
    if d % 32 == 0:
        codes = torch.zeros(2, m, heads, d // 2, dtype=torch.uint8, device="cuda")
        scales = torch.zeros(2, m, heads, d // 32, dtype=torch.uint8, device="cuda")
        near = x.contiguous()
        for i, t in enumerate((x, near)):
            kq.cache_write_mxfp4(torch.arange(m, device="cuda"), v=t, codes_v=codes[i], scales_v=scales[i])
        assert torch.equal(codes[0], codes[1]) and torch.equal(scales[0], scales[1])


def test_many_tokens_and_far_addresses(torch, kq):
    """Rows past 2^31 bytes of each tensor, in heads side by side and in tokens side by side."""
    m, heads, d = 40000, 17, 4 * 256  # 1.4 GB a tensor in bf16, and 2.8 with the stride below
    x = torch.empty(m, 2 * heads, d, dtype=torch.bfloat16, device="cuda")[:, ::2]
    tail = torch.randn(64, heads, d, device="cuda").to(torch.bfloat16)
    x.fill_(1.0)
    x[-64:] = tail
    rope = make_rope(torch, torch.Generator("cuda").manual_seed(1), m, 64, False)
    y = kq.headnorm_rope(x, eps=EPS, **call_args(rope))
    last = {**rope, "positions": rope["positions"][-64:].clone()}
    want, tol = ref.forward(tail, None, None, heads, EPS, last)
    layer_ref.assert_near(y[-64:], want, tol)
    del y
    out = torch.empty(heads, m, d, dtype=torch.bfloat16, device="cuda").transpose(0, 1)
    kq.headnorm_rope(x, eps=EPS, out=out, **call_args(rope))
    layer_ref.assert_near(out[-64:], want, tol)


# --- the cache -------------------------------------------------------------------------------
def make_cache(torch, g, slots, heads, d):
    return (torch.randint(0, 256, (slots, heads, d // 2), generator=g, device="cuda", dtype=torch.uint8),
            torch.randint(100, 140, (slots, heads, d // 32), generator=g, device="cuda", dtype=torch.uint8))


CACHES = [(1, 8, 128, 128, True), (64, 8, 128, 128, True), (7, 1, 32, 32, True), (5, 3, 32, 0, False), (9, 2, 64, 32, True),
          (33, 5, 96, 96, True), (4, 2, 160, 40, False), (3, 4, 256, 256, True), (2, 3, 1024, 1024, True),
          (3, 2, 992, 62, True), (500, 2, 64, 64, False), (1200, 8, 128, 128, True), (2100, 1, 32, 4, True)]


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("m,heads,d,rot,norm", CACHES)
def test_cache_write_and_read(torch, kq, m, heads, d, rot, norm, inter, dtype):
    dtype = getattr(torch, dtype)
    g = torch.Generator("cuda").manual_seed(m + d)
    kv = make_heads(torch, g, m, 2 * heads, d, dtype)
    k, v = kv[:, :heads], kv[:, heads:]
    weight = 1 + 0.2 * torch.randn(d, generator=g, device="cuda")
    rope = make_rope(torch, g, m, rot, inter)
    n = m + 21
    slots = torch.randperm(n, generator=g, device="cuda")[:m].contiguous()
    # padding: every seventh token is left out, below the cache or behind it
    for i, bad in zip(range(3, m, 7), [-1, n, -(1 << 62), (1 << 62), n + 5] * m):
        slots[i] = bad
    (ck, sk), (cv, sv) = make_cache(torch, g, n, heads, d), make_cache(torch, g, n, heads, d)
    before = [t.clone() for t in (ck, sk, cv, sv)]
    kq.cache_write_mxfp4(slots, k=k, codes_k=ck, scales_k=sk, v=v, codes_v=cv, scales_v=sv, norm=norm, weight=weight,
                         eps=EPS, **call_args(rope))
    in_cache = (slots >= 0) & (slots < n)
    at = slots[in_cache]
    # values: the quantizer's own bytes
    flat = v.reshape(m * heads, d).contiguous()
    c, s = kq.quantize_mxfp4(flat) if dtype == torch.bfloat16 else kq.quantize_mxfp4_f32(flat)
    assert torch.equal(cv[at], c.view(m, heads, d // 2)[in_cache])
    assert torch.equal(sv[at], s.view(m, heads, d // 32)[in_cache])
    y, tol = ref.forward(k, weight, weight, heads, EPS, rope, norm=norm)
    ref.assert_codes_near(ck[at], sk[at], y[in_cache], tol[in_cache], "keys")
    # no other slot is touched
    rest = torch.ones(n, dtype=torch.bool, device="cuda")
    rest[at] = False
    for t, b in zip((ck, sk, cv, sv), before):
        assert torch.equal(t[rest], b[rest])
    # keys or values alone
    for one in ("k", "v"):
        again = [t.clone() for t in before]
        kw = dict(k=k, codes_k=again[0], scales_k=again[1], norm=norm, weight=weight, eps=EPS, **call_args(rope)) \
            if one == "k" else dict(v=v, codes_v=again[2], scales_v=again[3])
        kq.cache_write_mxfp4(slots, **kw)
        for i, (a, b) in enumerate(zip(again, (ck, sk, cv, sv))):
            assert torch.equal(a, b if (i < 2) == (one == "k") else before[i])
    # read back: the decoder's own values, zeros for what is not there
    for codes, scales in ((ck, sk), (cv, sv)):
        got = kq.cache_read_mxfp4(slots, codes, scales, bf16=dtype == torch.bfloat16)
        full = kq.dequantize_mxfp4_bf16(codes.view(n * heads, -1), scales.view(n * heads, -1)).view(n, heads, d)
        want = torch.zeros(m, heads, d, dtype=dtype, device="cuda")
        want[in_cache] = full[at].to(dtype)
        assert torch.equal(got, want)


@pytest.mark.parametrize("heads,d,rot,dtype", [(2, 64, 64, "bfloat16"), (8, 128, 128, "bfloat16"), (3, 96, 32, "float32"),
                                               (1, 32, 32, "bfloat16")])
def test_cache_padding_may_hold_anything(torch, kq, heads, d, rot, dtype):
    """Padding tokens between the others, with NaN and infinities, the least and the greatest positions and slots of every
    wrong kind: the others' rows are those of a call without them."""
    g = torch.Generator("cuda").manual_seed(d)
    m, n = 150, 200
    k, v = (make_heads(torch, g, m, heads, d, getattr(torch, dtype)) for _ in range(2))
    slots = torch.randperm(n, generator=torch.Generator().manual_seed(d))[:m].cuda()
    rope = make_rope(torch, g, m, rot, False)
    pad = torch.arange(m, device="cuda") % 3 == 1
    bad = torch.tensor([-1, n, -2 ** 63, 2 ** 63 - 1, 2 ** 32, -(2 ** 32)], device="cuda")
    slots[pad] = bad[torch.arange(int(pad.sum()), device="cuda") % 6]
    junk = torch.tensor([math.nan, math.inf, -math.inf, torch.finfo(k.dtype).max], device="cuda").to(k.dtype)
    for t in (k, v):
        t[pad] = junk[torch.randint(0, 4, (int(pad.sum()), heads, d), generator=g, device="cuda")]
    rope["positions"][pad] = torch.tensor([-2 ** 63, 2 ** 63 - 1], device="cuda")[torch.arange(int(pad.sum()), device="cuda") % 2]
    weight = 1 + 0.1 * torch.randn(d, generator=g, device="cuda")

    def write(keep):
        codes = torch.full((2, n, heads, d // 2), 0x5A, dtype=torch.uint8, device="cuda")
        scales = torch.full((2, n, heads, d // 32), 0x5A, dtype=torch.uint8, device="cuda")
        args = {**call_args(rope), "positions": rope["positions"][keep].contiguous()}
        kq.cache_write_mxfp4(slots[keep].contiguous(), k=k[keep], codes_k=codes[0], scales_k=scales[0], v=v[keep],
                             codes_v=codes[1], scales_v=scales[1], norm=True, weight=weight, eps=EPS, **args)
        return codes, scales

    got, want = write(torch.ones_like(pad)), write(~pad)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    # wrong slots read as zeros
    back = kq.cache_read_mxfp4(slots, got[0][0], got[1][0])
    assert not back[pad].any() and bool((back[~pad] != 0).any())


def test_cache_read_every_scale_and_strides(torch, kq):
    """All scale bytes but NaN's with all codes, the same slot many times, rows apart."""
    codes = torch.arange(256, device="cuda").to(torch.uint8).repeat_interleave(16 * 4).view(256, 4, 16).contiguous()
    codes = codes.flip(0).contiguous()
    scales = torch.arange(255, -1, -1, device="cuda").clamp(max=254).to(torch.uint8).view(256, 1, 1).expand(256, 4, 1).contiguous()
    g = torch.Generator("cuda").manual_seed(2)
    codes ^= torch.randint(0, 256, codes.shape, generator=g, device="cuda", dtype=torch.uint8)
    slots = torch.randint(0, 256, (999,), generator=g, device="cuda")
    want = layer_ref.decode(codes.view(1024, 16), scales.view(1024, 1)).view(256, 4, 32)[slots]
    for dtype in (torch.bfloat16, torch.float32):
        for gap, shift, major in ((0, 0, False), (8, 8, False), (1, 1, False), (8, 0, True), (3, 2, True)):
            base, out = strided(torch, torch.zeros(999, 4, 32, dtype=dtype, device="cuda"), 4 * gap, gap, major, shift)
            base.fill_(math.nan)
            before = base.clone()
            kq.cache_read_mxfp4(slots, codes, scales, bf16=dtype == torch.bfloat16, out=out)
            # a value past the type's largest (levels of 4 and 6 at scale 254) is an infinity
            assert torch.equal(out.double(), want.to(dtype).double())
            out.fill_(math.nan)
            assert torch.equal(base.view(torch.uint8), before.view(torch.uint8))


def test_cache_past_32_bits(torch, kq):
    """A cache of more than 2^32 bytes of codes: its first and last slots."""
    heads, d = 8, 1024
    n = (1 << 32) // (heads * d // 2) + 100
    codes = torch.zeros(n, heads, d // 2, dtype=torch.uint8, device="cuda")
    scales = torch.zeros(n, heads, d // 32, dtype=torch.uint8, device="cuda")
    g = torch.Generator("cuda").manual_seed(8)
    v = make_heads(torch, g, 4, heads, d, torch.bfloat16)
    slots = torch.tensor([n - 1, 0, n - 50, n // 2], device="cuda")
    kq.cache_write_mxfp4(slots, v=v, codes_v=codes, scales_v=scales)
    c, s = kq.quantize_mxfp4(v.reshape(4 * heads, d))
    assert torch.equal(codes[slots], c.view(4, heads, -1)) and torch.equal(scales[slots], s.view(4, heads, -1))
    assert int((codes[1:100] != 0).sum()) == 0
    want = kq.dequantize_mxfp4_bf16(c, s).view(4, heads, d)
    assert torch.equal(kq.cache_read_mxfp4(slots, codes, scales), want)


def test_cache_streams_and_graphs(torch, kq):
    g = torch.Generator("cuda").manual_seed(12)
    m, heads, d, n = 40, 4, 128, 90
    k, v = (make_heads(torch, g, m, heads, d, torch.bfloat16) for _ in range(2))
    rope = make_rope(torch, g, m, d, False)
    slots = torch.randperm(n, generator=g, device="cuda")[:m].contiguous()
    caches = [make_cache(torch, g, n, heads, d) for _ in range(2)]

    def step(caches, stream=None):
        (ck, sk), (cv, sv) = caches
        kq.cache_write_mxfp4(slots, k=k, codes_k=ck, scales_k=sk, v=v, codes_v=cv, scales_v=sv, norm=True, eps=EPS,
                             stream=stream, **call_args(rope))
        return [kq.cache_read_mxfp4(slots, c, s, stream=stream) for c, s in caches]

    copies = [[(c.clone(), s.clone()) for c, s in caches] for _ in range(3)]
    want = step(caches)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [step(copies[i], s) for i, s in enumerate(streams)]
    torch.cuda.synchronize()
    for o in got:
        assert all(torch.equal(a, b) for a, b in zip(o, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(copies[2])
    for _ in range(3):
        k.copy_(make_heads(torch, g, m, heads, d, torch.bfloat16))
        slots.copy_(torch.randperm(n, generator=g, device="cuda")[:m])
        graph.replay()
        torch.cuda.synchronize()
        got = [o.clone() for o in out]
        want = step(caches)
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_refusals_of_the_binding(torch, kq):
    x = torch.zeros(4, 2, 64, device="cuda")
    freq, pos = torch.ones(32, dtype=torch.float64, device="cuda"), torch.arange(4, device="cuda")
    for kw, error in [
            (dict(x=x.half()), TypeError), (dict(x=x.cpu()), TypeError), (dict(x=x[0]), ValueError),
            (dict(x=x.transpose(1, 2)), ValueError), (dict(freq=freq.float(), positions=pos), TypeError),
            (dict(freq=freq, positions=pos.int()), TypeError), (dict(freq=freq), TypeError),
            (dict(freq=freq, positions=pos[:3]), ValueError), (dict(freq=freq, positions=pos.cpu()), ValueError),
            (dict(freq=freq, positions=pos.view(4, 1).repeat(1, 2)), ValueError),
            (dict(freq=freq, positions=pos.view(4, 1).repeat(1, 2), axis_pairs=(16, 15)), kq.KQError),
            (dict(freq=torch.ones(33, dtype=torch.float64, device="cuda"), positions=pos), kq.KQError),
            (dict(weight_q=torch.ones(63, device="cuda")), ValueError), (dict(q_heads=3), kq.KQError),
            (dict(eps=-1.0), kq.KQError), (dict(eps=math.nan), kq.KQError),
            (dict(out=torch.zeros(1, 1, 64, device="cuda").expand(4, 2, 64)), kq.KQError),
            (dict(out=x.bfloat16()), TypeError)]:
        with pytest.raises(error):
            kq.headnorm_rope(**{"x": x, **kw})
    with pytest.raises(ValueError):
        kq.headnorm_rope_backward(x)
    with pytest.raises(kq.KQError):
        kq.headnorm_rope_backward(x, x, workspace=torch.empty(0, dtype=torch.uint8, device="cuda"), q_heads=9)
    codes, scales = torch.zeros(9, 2, 32, dtype=torch.uint8, device="cuda"), torch.zeros(9, 2, 2, dtype=torch.uint8, device="cuda")
    slots = torch.arange(4, device="cuda")
    for kw, error in [(dict(slots=slots.int()), TypeError), (dict(slots=slots[:3]), ValueError), (dict(v=None), ValueError),
                      (dict(codes_v=codes[:, :1]), ValueError), (dict(scales_v=scales[:8]), ValueError),
                      (dict(codes_v=codes.int()), TypeError), (dict(v=x[:, :, :32]), ValueError)]:
        with pytest.raises(error):
            kq.cache_write_mxfp4(**{"slots": slots, "v": x, "codes_v": codes, "scales_v": scales, **kw})
    for kw, error in [(dict(slots=slots.int()), TypeError), (dict(scales=scales[:, :1]), ValueError),
                      (dict(out=torch.zeros(3, 2, 64, dtype=torch.bfloat16, device="cuda")), ValueError)]:
        with pytest.raises(error):
            kq.cache_read_mxfp4(**{"slots": slots, "codes": codes, "scales": scales, **kw})
