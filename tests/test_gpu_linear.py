"""GPU: the W4A4 product with bias, activation and residual in its epilogue, and that epilogue's
gradients, against 64-bit plain forms (tests/layer_ref.py), within bounds derived there."""
import pytest

from tests import layer_ref as ref

pytestmark = pytest.mark.gpu

ACTS = ["none", "relu", "silu", "gelu", "gelu_tanh"]


def case(msg):
    print("[case] " + msg, flush=True)


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


def gen(torch, seed):
    return torch.Generator("cuda").manual_seed(seed)


def operand(torch, kq, rows, k, seed, scale=1.0):
    """MXFP4 codes and scales of normal values."""
    if k == 0 or rows == 0:
        return (torch.empty((rows, k // 2), dtype=torch.uint8, device="cuda"),
                torch.empty((rows, k // 32), dtype=torch.uint8, device="cuda"))
    x = torch.randn(rows, k, generator=gen(torch, seed), device="cuda") * scale
    return kq.quantize_mxfp4_f32(x)


def check(torch, kq, m, n, k, name, dt, packed, bias=True, residual=True, seed=0, pad=0):
    dtype = getattr(torch, dt)
    case("linear %dx%dx%d %s %s packed=%d" % (m, n, k, name, dt, packed))
    ca, sa = operand(torch, kq, m, k, seed + 1)
    cw, sw = operand(torch, kq, n, k, seed + 2, 1.0 if k == 0 else k ** -0.5)
    b = torch.randn(n, generator=gen(torch, seed + 3), device="cuda") if bias else None

    def room():
        buf = torch.full((m, n + pad), float("nan"), dtype=dtype, device="cuda")
        return buf, buf[:, :n]

    res = None
    if residual:
        _, res = room()
        res.copy_(torch.randn(m, n, generator=gen(torch, seed + 4), device="cuda"))
    pa, pw = (kq.pack_mxfp4_scales(sa), kq.pack_mxfp4_scales(sw)) if packed else (sa, sw)
    (obuf, out), (zbuf, pre) = room(), room()
    kq.mxfp4_linear(ca, pa, cw, pw, bias=b, act=name, residual=res, out=out, pre=pre, bf16=dt == "bfloat16",
                    packed=packed)
    o, z, o_tol, z_tol = ref.linear(ca, sa, cw, sw, b, name, res)
    ref.assert_near(pre, z, z_tol, "z")
    ref.assert_near(out, o, o_tol, "out")
    assert int(obuf.isnan().sum()) == m * pad and int(zbuf.isnan().sum()) == m * pad  # the padding is left alone
    alone = kq.mxfp4_linear(ca, pa, cw, pw, bias=b, act=name, residual=res, bf16=dt == "bfloat16", packed=packed)
    assert torch.equal(alone, out)  # z asked for or not, padded or not, twice: the same output


# one token, a few, one past and one short of a tile; k of one block, of part of a stage, of many; odd n
SMALL = [(1, 16, 32), (1, 1, 64), (2, 33, 96), (7, 100, 1152), (16, 256, 512), (17, 130, 4096), (1, 1000, 2080),
         (33, 515, 288), (45, 1000, 1152), (64, 64, 2048), (65, 257, 640), (130, 300, 1056), (250, 129, 4608),
         (1, 16384, 256), (3, 5, 8192)]


@pytest.mark.parametrize("dt", ["bfloat16", "float32"])
@pytest.mark.parametrize("m,n,k", SMALL)
def test_few_rows(torch, kq, m, n, k, dt):
    for i, packed in enumerate([False, True] if k % 256 == 0 else [False]):
        check(torch, kq, m, n, k, ACTS[(m + n) % 5], dt, packed, seed=m)
        check(torch, kq, m, n, k, ACTS[(m + n + 1) % 5], dt, packed, bias=False, residual=i == 0, seed=n, pad=3)


# whole and ragged tiles of the many-row kernel, k of whole stages, of half ones, of neither
LARGE = [(256, 256, 256), (1024, 4096, 512), (700, 1300, 1152), (2048, 2048, 384), (1111, 2222, 768),
         (3000, 4104, 128), (513, 8191, 256), (4096, 520, 1056), (5000, 1024, 96)]


@pytest.mark.parametrize("dt", ["bfloat16", "float32"])
@pytest.mark.parametrize("m,n,k", LARGE)
def test_many_rows(torch, kq, m, n, k, dt):
    for packed in [False, True] if k % 256 == 0 else [False]:
        check(torch, kq, m, n, k, ACTS[(m + k // 32) % 5], dt, packed, seed=m, pad=8 * packed)


# one ragged product or more for every kernel the choice knows on 256 compute units (16 x 16, 16 x 32 and
# 32 x 32 tiles with split k; 64 x 64 four and two stages deep, 128 x 128, 256 x 256 through LDS), each with a
# k of whole stages (either layout), of a half stage and of single blocks as far as it takes them
EVERY = [(250, 129, 4608), (20, 4095, 512), (64, 4001, 1184), (60, 3901, 2304), (100, 4100, 2080), (130, 4093, 4096),
         (200, 4093, 1152), (600, 4099, 1024), (300, 3000, 96), (2050, 1154, 2304), (2050, 1155, 2336), (4100, 5000, 544),
         (3000, 4000, 1920), (1500, 3333, 4096), (1500, 3336, 3968), (2048, 4096, 1152)]


@pytest.mark.parametrize("m,n,k", EVERY)
def test_every_kernel(torch, kq, m, n, k):
    for i, packed in enumerate([False, True] if k % 256 == 0 else [False]):
        dt = ("bfloat16", "float32")[(m + k // 32 + i) % 2]
        check(torch, kq, m, n, k, ACTS[(n + i) % 5], dt, packed, seed=k, pad=(0, 8, 5)[m % 3])


# last tiles of one row and one column, whose code buffers are shorter than the stages that are loaded ahead
@pytest.mark.parametrize("m,n,k", [(65, 4033, 32), (65, 4033, 256), (129, 4033, 1056), (257, 4033, 288), (1537, 2561, 96),
                                   (1537, 2561, 1280)])
def test_one_row_in_the_last_tile(torch, kq, m, n, k):
    check(torch, kq, m, n, k, "silu", "bfloat16", False, seed=m)


@pytest.mark.parametrize("m,n,k", [(9, 300, 512), (60, 3901, 2304), (600, 4099, 1024), (2050, 1154, 2304)])
def test_scales_at_any_address(torch, kq, m, n, k):
    """MX-layout scales need no alignment: at odd addresses, the same output (bytes 1 and 3 into a
    buffer), whichever kernel runs."""
    ca, sa = operand(torch, kq, m, k, 1)
    cw, sw = operand(torch, kq, n, k, 2, k ** -0.5)
    want = kq.mxfp4_linear(ca, sa, cw, sw, act="relu", bf16=False)

    def moved(s, by):
        buf = torch.empty(s.numel() + by, dtype=torch.uint8, device="cuda")
        v = buf[by:].view(s.shape)
        v.copy_(s)
        return v

    o, z, o_tol, z_tol = ref.linear(ca, sa, cw, sw, None, "relu", None)
    for by_a, by_w in ((1, 3), (0, 1), (2, 0)):
        got = kq.mxfp4_linear(ca, moved(sa, by_a), cw, moved(sw, by_w), act="relu", bf16=False)
        ref.assert_near(got, o, o_tol)
    ref.assert_near(want, o, o_tol)


@pytest.mark.parametrize("name", ACTS)
@pytest.mark.parametrize("dt", ["bfloat16", "float32"])
def test_activations(torch, kq, name, dt):
    """Every activation over a wide range of z (the bias spreads it), on both kernels."""
    for m in (5, 1030):
        n, k = 1024, 256
        ca, sa = operand(torch, kq, m, k, 1)
        cw, sw = operand(torch, kq, n, k, 2, k ** -0.5)
        b = torch.linspace(-12, 12, n, device="cuda")
        out, pre = kq.mxfp4_linear(ca, sa, cw, sw, bias=b, act=name, bf16=dt == "bfloat16", want_pre=True)
        o, z, o_tol, z_tol = ref.linear(ca, sa, cw, sw, b, name, None)
        ref.assert_near(pre, z, z_tol, "z")
        ref.assert_near(out, o, o_tol, "out")


def test_no_inner_dimension_and_empty(torch, kq):
    """k = 0: act(bias) + residual; no rows or columns: nothing."""
    check(torch, kq, 5, 40, 0, "silu", "float32", False)
    check(torch, kq, 600, 700, 0, "gelu", "bfloat16", True)
    for m, n in ((0, 8), (8, 0), (0, 0)):
        ca, sa = operand(torch, kq, m, 64, 1)
        cw, sw = operand(torch, kq, n, 64, 2)
        assert kq.mxfp4_linear(ca, sa, cw, sw).shape == (m, n)


@pytest.mark.parametrize("m,n", [(5, 40), (40, 72), (200, 4100), (1030, 4000)])
def test_no_inner_dimension_packed(torch, kq, m, n):
    """k = 0 is a multiple of 256 too: O = act(bias) + residual whatever the scales' layout, in every tile."""
    case("k = 0 packed %dx%d" % (m, n))
    none = lambda rows: torch.empty((rows, 0), dtype=torch.uint8, device="cuda")
    b = torch.randn(n, generator=gen(torch, 1), device="cuda")
    res = torch.randn(m, n, generator=gen(torch, 2), device="cuda")
    args = (none(m), none(m), none(n), none(n))
    out, pre = kq.mxfp4_linear(*args, bias=b, act="relu", residual=res, bf16=False, packed=True, want_pre=True)
    assert torch.equal(pre, b.expand(m, n)) and torch.equal(out, b.clamp(min=0) + res)
    assert torch.equal(out, kq.mxfp4_linear(*args, bias=b, act="relu", residual=res, bf16=False))


def test_matches_plain_product(torch, kq):
    """Without bias, activation and residual: the product's own fp32 sums, rounded once for bf16."""
    ca, sa = operand(torch, kq, 1024, 768, 1)
    cw, sw = operand(torch, kq, 2048, 768, 2)
    pa, pw = kq.pack_mxfp4_scales(sa), kq.pack_mxfp4_scales(sw)
    want = kq.mxfp4_gemm_packed(ca, pa, cw, pw)
    for packed, a, w in ((True, pa, pw), (False, sa, sw)):
        f32 = kq.mxfp4_linear(ca, a, cw, w, bf16=False, packed=packed)
        o, z, o_tol, z_tol = ref.linear(ca, sa, cw, sw, None, "none", None)
        ref.assert_near(f32, o, o_tol)
        assert bool(((f32 - want).abs().double() <= 2 * z_tol).all())
        assert torch.equal(kq.mxfp4_linear(ca, a, cw, w, packed=packed), f32.bfloat16())


def test_extreme_scales(torch, kq):
    """Scale bytes 0 .. 2 against 250 .. 254, whose products are in range, and zero codes."""
    for m in (3, 520):
        n, k = 300, 512
        g = gen(torch, 5)
        ca = torch.randint(0, 256, (m, k // 2), generator=g, device="cuda", dtype=torch.uint8)
        cw = torch.randint(0, 256, (n, k // 2), generator=g, device="cuda", dtype=torch.uint8)
        sa = torch.randint(0, 3, (m, k // 32), generator=g, device="cuda", dtype=torch.uint8)
        sw = torch.randint(250, 255, (n, k // 32), generator=g, device="cuda", dtype=torch.uint8)
        ca[1] = 0
        got = kq.mxfp4_linear(ca, sa, cw, sw, bf16=False)
        o, z, o_tol, z_tol = ref.linear(ca, sa, cw, sw, None, "none", None)
        ref.assert_near(got, o, o_tol)
        assert not bool(got[1].any())


@pytest.mark.parametrize("name", ACTS)
@pytest.mark.parametrize("dt", ["bfloat16", "float32"])
@pytest.mark.parametrize("m,n", [(1, 1), (1, 4096), (16, 100), (17, 64), (301, 1003), (40, 4608), (9000, 72), (700, 2056)])
def test_backward(torch, kq, m, n, dt, name):
    dtype = getattr(torch, dt)
    case("linear_grad %dx%d %s %s" % (m, n, dt, name))
    dout = torch.randn(m, n, generator=gen(torch, 1), device="cuda").to(dtype)
    z = (2.5 * torch.randn(m, n, generator=gen(torch, 2), device="cuda")).to(dtype)
    got = kq.mxfp4_linear_backward(dout, z, act=name)
    want, tol = ref.linear_grad(dout, z, name)
    for g, v, t, what in zip(got, want, tol, ("dz", "dbias")):
        ref.assert_near(g, v, t, what)
    again = kq.mxfp4_linear_backward(dout, z, act=name)
    assert torch.equal(got[0], again[0]) and torch.equal(got[1], again[1])
    if name == "none":
        alone = kq.mxfp4_linear_backward(dout)
        assert torch.equal(alone[0], got[0]) and torch.equal(alone[1], got[1])


@pytest.mark.parametrize("dt", ["bfloat16", "float32"])
def test_backward_streamed(torch, kq, dt):
    """128 MiB and more (non-temporal accesses), an odd number of rows and of strips."""
    dtype = getattr(torch, dt)
    m, n = 8311, 2728
    dout = torch.randn(m, n, generator=gen(torch, 1), device="cuda").to(dtype)
    z = torch.randn(m, n, generator=gen(torch, 2), device="cuda").to(dtype)
    got = kq.mxfp4_linear_backward(dout, z, act="gelu_tanh")
    want, tol = ref.linear_grad(dout, z, "gelu_tanh")
    for g, v, t in zip(got, want, tol):
        ref.assert_near(g, v, t)


@pytest.mark.parametrize("m,n", [(8311, 2729), (1, 511), (3, 513), (1000, 4001), (5, 1025)])
@pytest.mark.parametrize("dt", ["bfloat16", "float32"])
def test_backward_odd_widths(torch, kq, m, n, dt):
    """Rows that are no whole 16 bytes, streamed ones too: a lane takes every 64th column."""
    dtype = getattr(torch, dt)
    dout = torch.randn(m, n, generator=gen(torch, m), device="cuda").to(dtype)
    z = torch.randn(m, n, generator=gen(torch, n), device="cuda").to(dtype)
    for name in ("none", "silu"):
        got = kq.mxfp4_linear_backward(dout, z, act=name)
        want, tol = ref.linear_grad(dout, z, name)
        for g, v, t in zip(got, want, tol):
            ref.assert_near(g, v, t)


@pytest.mark.parametrize("dt", ["bfloat16", "float32"])
@pytest.mark.parametrize("m,n", [(4100, 16384 * 2), (4099, 32771)])
def test_residual_past_the_cache(torch, kq, m, n, dt):
    """A residual of 256 MiB and more (read non-temporally), whole 16-byte rows and odd ones."""
    check(torch, kq, m, n, 256, "relu", dt, True, seed=m)


@pytest.mark.parametrize("m,n,k", [(1, 512, 256), (64, 4001, 1184), (100, 4100, 2080), (2050, 1155, 2336), (1500, 3336, 3968)])
def test_residual_in_place(torch, kq, m, n, k):
    """O = act(z) + O on every family of kernels, aligned rows and ragged ones."""
    ca, sa = operand(torch, kq, m, k, 1)
    cw, sw = operand(torch, kq, n, k, 2, k ** -0.5)
    for bf16 in (True, False):
        x = torch.randn(m, n, generator=gen(torch, 4), device="cuda").to(torch.bfloat16 if bf16 else torch.float32)
        want = kq.mxfp4_linear(ca, sa, cw, sw, act="silu", residual=x, bf16=bf16)
        got = kq.mxfp4_linear(ca, sa, cw, sw, act="silu", residual=x, out=x, bf16=bf16)
        assert got is x and torch.equal(x, want)


def test_outputs_past_32_bits(torch, kq):
    """Rows of the outputs, the residual and the gradients 2^20 elements apart: offsets past 2^31."""
    ld, m, n, k = 1 << 20, 2300, 136, 256
    buf = torch.empty(m * ld, dtype=torch.bfloat16, device="cuda").view(m, ld)
    ca, sa = operand(torch, kq, m, k, 1)
    cw, sw = operand(torch, kq, n, k, 2, k ** -0.5)
    res, out, pre = buf[:, 0:n], buf[:, 4096:4096 + n], buf[:, 8192:8192 + n]
    res.copy_(torch.randn(m, n, generator=gen(torch, 3), device="cuda"))
    kq.mxfp4_linear(ca, sa, cw, sw, act="silu", residual=res, out=out, pre=pre)
    o, z, o_tol, z_tol = ref.linear(ca, sa, cw, sw, None, "silu", res)
    ref.assert_near(pre, z, z_tol, "z")
    ref.assert_near(out, o, o_tol, "out")
    for lo in (16384, 16385):  # the vector path and the general one
        dz, dbias = kq.mxfp4_linear_backward(res, pre, act="silu", dz=buf[:, lo:lo + n])
        want, tol = ref.linear_grad(res, pre, "silu")
        ref.assert_near(dz, want[0], tol[0])
        ref.assert_near(dbias, want[1], tol[1])


@pytest.mark.parametrize("extra,offset", [(8, 0), (3, 0), (0, 1)])
def test_backward_strides_and_alignment(torch, kq, extra, offset):
    m, n = 50, 712
    for dtype in (torch.bfloat16, torch.float32):
        def place(v):
            buf = torch.full((m * (n + extra) + offset + 64,), float("nan"), dtype=dtype, device="cuda")
            view = buf[offset:offset + m * (n + extra)].view(m, n + extra)[:, :n]
            view.copy_(v)
            return view, buf

        dout, _ = place(torch.randn(m, n, generator=gen(torch, 1), device="cuda"))
        z, _ = place(torch.randn(m, n, generator=gen(torch, 2), device="cuda"))
        dz, buf = place(torch.zeros(m, n, device="cuda"))
        got = kq.mxfp4_linear_backward(dout, z, act="gelu", dz=dz)
        want, tol = ref.linear_grad(dout, z, "gelu")
        for g, v, t in zip(got, want, tol):
            ref.assert_near(g, v, t)
        assert int(buf.isnan().sum()) == buf.numel() - m * n


def test_backward_far_arguments(torch, kq):
    """Slopes where the activation is saturated, and far beyond: finite, 0 or 1 times dout."""
    z = torch.tensor([[-1e30, -3e19, -200.0, -60.0, 0.0, 60.0, 200.0, 3e19, 1e30]], device="cuda")
    d = torch.ones_like(z)
    for name in ACTS:
        dz = kq.mxfp4_linear_backward(d, z, act=name)[0]
        assert bool(dz.isfinite().all()), name
        if name != "none":
            assert not bool((dz[0, :4].abs() > 1e-20).any()) and torch.equal(dz[0, 5:], d[0, 5:]), name


def test_refusals(torch, kq):
    ca, sa = operand(torch, kq, 4, 64, 1)
    cw, sw = operand(torch, kq, 8, 64, 2)
    with pytest.raises(ValueError):
        kq.mxfp4_linear(ca, sa, cw, sw, act="tanh")
    with pytest.raises(ValueError):
        kq.mxfp4_linear(ca, sa, cw[:, :16], sw)
    with pytest.raises(ValueError):
        kq.mxfp4_linear(ca, sa[:3], cw, sw)
    with pytest.raises(ValueError):
        kq.mxfp4_linear(ca, sa, cw, sw, bias=torch.zeros(9, device="cuda"))
    with pytest.raises(TypeError):
        kq.mxfp4_linear(ca, sa, cw, sw, residual=torch.zeros(4, 8, device="cuda"))  # fp32 beside a bf16 output
    with pytest.raises(ValueError):
        kq.mxfp4_linear(ca, sa, cw, sw, out=torch.zeros(4, 9, device="cuda", dtype=torch.bfloat16))
    with pytest.raises(kq.KQError):
        kq.mxfp4_linear(ca, sa, cw, sw, packed=True)  # k is no whole number of stages
    x = torch.zeros(4, 8, device="cuda")
    with pytest.raises(ValueError):
        kq.mxfp4_linear_backward(x, None, act="relu")
    with pytest.raises(TypeError):
        kq.mxfp4_linear_backward(x, x.bfloat16(), act="relu")
    with pytest.raises(TypeError):
        kq.mxfp4_linear_backward(x.double(), x, act="relu")


@pytest.mark.parametrize("m,n", [(5, 0), (0, 0), (0, 5)])
def test_backward_of_nothing(torch, kq, m, n):
    """No columns: an empty dz and an empty dbias; no rows: dbias of zeros."""
    x = torch.empty((m, n), device="cuda")
    dz, dbias = kq.mxfp4_linear_backward(x, x, act="silu")
    assert dz.shape == (m, n) and dbias.shape == (n,) and not bool(dbias.any())


def with_activation(torch, kq, z, name, dt):
    """act(z) and its slope at given fp32 z: k = 0 makes z the bias; the slope is dz of dout = 1."""
    n = z.numel()
    none = [torch.empty((r, 0), dtype=torch.uint8, device="cuda") for r in (1, 1, n, n)]
    out = kq.mxfp4_linear(*none, bias=z, act=name, bf16=dt == "bfloat16")[0]
    slope = kq.mxfp4_linear_backward(torch.ones(1, n, device="cuda"), z.view(1, n), act=name)[0][0]
    return out, slope


@pytest.mark.parametrize("dt", ["bfloat16", "float32"])
def test_gelu_is_good_to_its_last_bits(torch, kq, dt):
    """gelu keeps a relative error where it vanishes: P(z) to 13 u of itself (t to 2 u, times at most 2.3 = the
    slope of log R in log t: 4.6; the polynomial 0.6 of its fit and 1.5 of rounding; the exponential 2 u of the
    instruction and 2 of its correction; two products; 1 - tail adds a rounding), and one more for the product
    with z. bf16 outputs: the fit 30 u, t to 3 u times 2.3, the polynomial and its products 4, the exponential 2
    and its exponent's roundings 1.2 z^2, before the output's own. The slope P + z phi adds the exponential's 4 u and three products' u of z phi, and its own sum's."""
    z = torch.cat((torch.linspace(-13, 13, 40001), torch.linspace(-1e-3, 1e-3, 2001))).cuda()
    out, slope = with_activation(torch, kq, z, "gelu", dt)
    e = z.double()
    p = 0.5 * torch.erfc(-e * 0.5 ** 0.5)
    u = 14 if dt == "float32" else 46 + 1.2 * e * e
    ref.assert_near(out, e * p, u * ref.U * (e * p).abs(), "gelu")
    zphi = e * torch.exp(-e * e / 2) * 0.3989422804014327
    ref.assert_near(slope, p + zphi, 13 * ref.U * p + 8 * ref.U * zphi.abs() + ref.U * (p + zphi).abs(), "slope")


@pytest.mark.parametrize("name,low", [("silu", -80.0), ("gelu_tanh", -9.0)])
def test_logistic_error_grows_with_its_exponent_alone(torch, kq, name, low):
    """silu and gelu_tanh in fp32 relative to their values: the logistic's exponent y is off by 1.3 u of
    itself in silu (the constant 0.23 u, the product 1 u), by 6 u in gelu_tanh (constants 1 and 3, z^2, the sum
    and the product 1 each), which exp(y) multiplies by |y|; exp2 2 u, 1 + e 1 u, the reciprocal 2 u, z s 1 u."""
    z = torch.linspace(low, 30.0, 30011).cuda()
    out, _ = with_activation(torch, kq, z, name, "float32")
    e = z.double()
    y = -e if name == "silu" else -2 * (2 / torch.pi) ** 0.5 * (e + 0.044715 * e ** 3)
    want = e / (1 + torch.exp(y))
    ref.assert_near(out, want, ((1.3 if name == "silu" else 6) * y.clamp(min=0) + 7) * ref.U * want.abs(), name)


# products of the 256 x 256 kernel (tests/test_linear_choice.py holds them to it): tiles computed whole and as
# halves, rows of whole 16 bytes and not, ragged last tiles, k of whole stages (either layout) and with a half one
BIG = [(4096, 4096, 4096), (4100, 4360, 4096), (4093, 4103, 2304), (3333, 4104, 4096), (4096, 4096, 768),
       (4096, 4096, 3968), (4100, 4363, 1920), (4100, 4360, 1920), (4100, 8200, 1152)]
BIG_IN_PLACE = [(4100, 4360, 4096), (4093, 4103, 2304)]
# with outputs of 256 MiB and more, whose residual is read non-temporally
BIG_STREAMED = [(8192, 16384, 1024, "bfloat16"), (8192, 8192, 1024, "float32"), (8200, 16391, 1024, "bfloat16")]

# 32 x 32 tiles of ragged products with a partial last stage
PART = [(50, 4001, 1184), (90, 2050, 800)]


@pytest.mark.parametrize("dt", ["bfloat16", "float32"])
@pytest.mark.parametrize("m,n,k", PART)
def test_partial_stages(torch, kq, m, n, k, dt):
    check(torch, kq, m, n, k, "silu", dt, False, seed=k, pad=5)


@pytest.mark.parametrize("dt", ["bfloat16", "float32"])
@pytest.mark.parametrize("m,n,k", BIG)
def test_big_tiles(torch, kq, m, n, k, dt):
    for i, packed in enumerate([False, True] if k % 256 == 0 else [False]):
        check(torch, kq, m, n, k, ACTS[(m + k // 128 + i) % 5], dt, packed, seed=k, pad=(0, 8, 5)[(m + i) % 3])


@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("m,n,k", BIG_IN_PLACE)
def test_big_residual_in_place(torch, kq, m, n, k, packed):
    ca, sa = operand(torch, kq, m, k, 1)
    cw, sw = operand(torch, kq, n, k, 2, k ** -0.5)
    if packed:
        sa, sw = kq.pack_mxfp4_scales(sa), kq.pack_mxfp4_scales(sw)
    for bf16 in (True, False):
        x = torch.randn(m, n, generator=gen(torch, 4), device="cuda").to(torch.bfloat16 if bf16 else torch.float32)
        want = kq.mxfp4_linear(ca, sa, cw, sw, act="silu", residual=x, bf16=bf16, packed=packed)
        got = kq.mxfp4_linear(ca, sa, cw, sw, act="silu", residual=x, out=x, bf16=bf16, packed=packed)
        assert got is x and torch.equal(x, want)


@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("m,n,k,dt", BIG_STREAMED)
def test_big_residual_past_the_cache(torch, kq, m, n, k, dt, packed):
    check(torch, kq, m, n, k, "relu", dt, packed, seed=m)


@pytest.mark.parametrize("dt", ["bfloat16", "float32"])
@pytest.mark.parametrize("m", [1, 2, 3, 5, 17, 33, 127, 255, 1023, 1025, 1027, 2053, 9001])
@pytest.mark.parametrize("n", [8, 72, 511, 1032, 4101])
def test_backward_sums_every_row_once(torch, kq, m, n, dt):
    """With dout small integers dbias is an integer without any rounding (relu keeps or drops whole ones), below
    2^24: a row left out or counted twice shows in every column."""
    sums_every_row_once(torch, kq, m, n, dt)


@pytest.mark.parametrize("dt", ["bfloat16", "float32"])
@pytest.mark.parametrize("m,n", [(8311, 2728), (8311, 2729), (1033, 21680), (1033, 21681), (45013, 520)])
def test_backward_sums_every_row_once_streamed(torch, kq, m, n, dt):
    sums_every_row_once(torch, kq, m, n, dt)


def sums_every_row_once(torch, kq, m, n, dt):
    dtype = getattr(torch, dt)
    v = torch.randint(1, 4, (m, n), generator=gen(torch, m), device="cuda")
    z = torch.randn(m, n, generator=gen(torch, n), device="cuda").to(dtype)
    dout = torch.where(torch.rand(m, n, generator=gen(torch, m + n), device="cuda") < 0.5, -v, v).to(dtype)
    dz, dbias = kq.mxfp4_linear_backward(dout)
    assert torch.equal(dz, dout) and torch.equal(dbias.double(), dout.double().sum(0))
    dz, dbias = kq.mxfp4_linear_backward(dout, z, act="relu")
    want = torch.where(z > 0, dout, torch.zeros_like(dout))
    assert torch.equal(dz, want) and torch.equal(dbias.double(), want.double().sum(0))


# a product for each kernel, with rows of O of whole 16 bytes
PLACES = [(5, 512, 512), (40, 4096, 512), (60, 4096, 2304), (130, 4096, 4096), (600, 4096, 1024), (2050, 1160, 2304),
          (4096, 4096, 768)]


@pytest.mark.parametrize("dt", ["bfloat16", "float32"])
@pytest.mark.parametrize("m,n,k", PLACES)
def test_operands_at_unlike_addresses(torch, kq, m, n, k, dt):
    """Residual, output, z and bias each with a row stride and an address of its own, aligned as their elements at
    least, in every combination of one that is not 16-byte aligned: the same bits as with all of them aligned."""
    dtype, g = getattr(torch, dt), gen(torch, k)
    ca, sa = operand(torch, kq, m, k, 1)
    cw, sw = operand(torch, kq, n, k, 2, k ** -0.5)
    res0 = torch.randn(m, n, generator=g, device="cuda").to(dtype)
    bias0 = torch.randn(n, generator=g, device="cuda")
    want, pre0 = kq.mxfp4_linear(ca, sa, cw, sw, bias=bias0, act="gelu", residual=res0, bf16=dt == "bfloat16",
                                 want_pre=True)

    def place(extra, offset):
        buf = torch.full((m * (n + extra) + offset,), float("nan"), dtype=dtype, device="cuda")
        return buf, buf[offset:].view(m, n + extra)[:, :n]

    for odd in ("none", "residual", "out", "pre", "bias", "all"):
        at = lambda name: (7, 3) if odd in (name, "all") else (16, 0)
        _, res = place(*at("residual"))
        res.copy_(res0)
        (obuf, out), (zbuf, pre) = place(*at("out")), place(*at("pre"))
        bias = torch.empty(n + 3, device="cuda")[at("bias")[1]:][:n]
        bias.copy_(bias0)
        kq.mxfp4_linear(ca, sa, cw, sw, bias=bias, act="gelu", residual=res, out=out, pre=pre, bf16=dt == "bfloat16")
        assert torch.equal(out, want) and torch.equal(pre, pre0), odd
        assert int(obuf.isnan().sum()) == obuf.numel() - m * n and int(zbuf.isnan().sum()) == zbuf.numel() - m * n


@pytest.mark.parametrize("m,n,k", [(40, 4096, 512), (600, 4096, 1024), (2050, 1160, 2304), (4096, 4096, 768)])
def test_packed_scales_8_byte_aligned(torch, kq, m, n, k):
    """Packed scales need 8 bytes of alignment; the 256 x 256 kernel, which wants 16, is passed over without them."""
    ca, sa = operand(torch, kq, m, k, 1)
    cw, sw = operand(torch, kq, n, k, 2, k ** -0.5)
    pa, pw = kq.pack_mxfp4_scales(sa), kq.pack_mxfp4_scales(sw)
    o, z, o_tol, z_tol = ref.linear(ca, sa, cw, sw, None, "silu", None)

    def moved(s, by):
        v = torch.empty(s.numel() + by, dtype=torch.uint8, device="cuda")[by:].view(s.shape)
        v.copy_(s)
        return v

    for by_a, by_w in ((0, 0), (8, 0), (0, 8), (8, 8)):
        ref.assert_near(kq.mxfp4_linear(ca, moved(pa, by_a), cw, moved(pw, by_w), act="silu", bf16=False, packed=True), o, o_tol)
    with pytest.raises(kq.KQError):
        kq.mxfp4_linear(ca, moved(pa, 4), cw, pw, packed=True)


@pytest.mark.parametrize("m,n,k", [(4100, 4360, 1920), (4096, 4096, 768)])
def test_big_tiles_with_scales_at_any_address(torch, kq, m, n, k):
    """MX scales 4-byte aligned stay on the 256 x 256 kernel, the same bits; at other addresses another one runs."""
    ca, sa = operand(torch, kq, m, k, 1)
    cw, sw = operand(torch, kq, n, k, 2, k ** -0.5)
    want = kq.mxfp4_linear(ca, sa, cw, sw, act="silu", bf16=False)
    o, z, o_tol, z_tol = ref.linear(ca, sa, cw, sw, None, "silu", None)
    ref.assert_near(want, o, o_tol)
    for by in (4, 12, 1, 2):
        a = torch.empty(sa.numel() + by, dtype=torch.uint8, device="cuda")[by:].view(sa.shape)
        a.copy_(sa)
        got = kq.mxfp4_linear(ca, a, cw, sw, act="silu", bf16=False)
        if by % 4 == 0:
            assert torch.equal(got, want)
        ref.assert_near(got, o, o_tol)


@pytest.mark.parametrize("dt", ["bfloat16", "float32"])
def test_far_arguments(torch, kq, dt):
    """Activations where they are saturated and far beyond: 0 or z itself; NaN stays NaN, and alone."""
    far = torch.tensor([-1e30, -3e19, -200.0, -105.0, 0.0, 60.0, 200.0, 3e19, 1e30], device="cuda")
    z = torch.cat((far, torch.full((1,), float("nan"), device="cuda"), far))
    n = far.numel()
    for name in ACTS[1:]:
        out, slope = with_activation(torch, kq, z, name, dt)
        assert bool(out[n].isnan()) and int(out.isnan().sum()) == 1, name
        assert int(slope.isnan().sum()) == (name != "relu"), name  # z > 0 is false for NaN: relu's slope is 0
        want = torch.where(far > 0, far, 0 * far).to(out.dtype)
        for part in (out[:n], out[n + 1:]):
            assert bool(((part - want).abs() <= 1e-30).all()) and torch.equal(part[5:], want[5:]), name
