"""GPU: layer norm, its gradients and the norm straight into the MXFP4 quantizer against 64-bit plain
forms (tests/layer_ref.py), within bounds derived there."""
import numpy as np
import pytest

import synth
from tests import layer_ref as ref
from tests import parity

pytestmark = pytest.mark.gpu

EPS = 1e-5


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


def rand(torch, *shape, seed, scale=1.0, shift=0.0, dtype=None):
    g = torch.Generator("cuda").manual_seed(seed)
    x = torch.randn(*shape, generator=g, device="cuda") * scale + shift
    return x if dtype is None else x.to(dtype)


def strided(torch, x, extra, offset=0):
    """x inside a wider buffer of NaN: row stride columns + extra, starting `offset` elements in."""
    m, d = x.shape
    buf = torch.full((m * (d + extra) + offset + 64,), float("nan"), dtype=x.dtype, device="cuda")
    view = buf[offset:offset + m * (d + extra)].view(m, d + extra)[:, :d]
    view.copy_(x)
    return view, buf


# (m, d): one element, odd widths, whole and partial vectors, one and several waves per row, rows beyond
# every register-resident width, more rows than workgroups in flight
SHAPES = [(1, 1), (1, 7), (3, 8), (5, 31), (2, 64), (300, 40), (4, 520), (37, 1152), (9, 4096), (2, 4104), (3, 8200),
          (2, 16384), (2, 40000), (1, 70001), (5000, 264)]


@pytest.mark.parametrize("dt", ["bfloat16", "float32"])
@pytest.mark.parametrize("m,d", SHAPES)
def test_forward(torch, kq, m, d, dt):
    dtype = getattr(torch, dt)
    case("norm %dx%d %s" % (m, d, dt))
    x = rand(torch, m, d, seed=m + d, scale=2.0, shift=0.5, dtype=dtype)
    w, b = rand(torch, d, seed=1, shift=1.0), rand(torch, d, seed=2)
    for ww, bb in ((w, b), (None, b), (w, None), (None, None)):
        y, mean, rstd = kq.layernorm(x, ww, bb, eps=EPS, stats=True)
        y0, mu, rs, y_tol, mu_tol, rs_tol = ref.norm(x, ww, bb, EPS)
        ref.assert_near(y, y0, y_tol, "y")
        ref.assert_near(mean, mu, mu_tol, "mean")
        ref.assert_near(rstd, rs, rs * rs_tol, "rstd")
    assert torch.equal(kq.layernorm(x, None, None, eps=EPS), y)  # without the statistics: the same


@pytest.mark.parametrize("dt", ["bfloat16", "float32"])
@pytest.mark.parametrize("extra,offset", [(8, 0), (3, 0), (0, 1), (16, 8)])
def test_strides_and_alignment(torch, kq, dt, extra, offset):
    """Padded and misaligned rows: the padding (NaN) is neither read nor written."""
    dtype = getattr(torch, dt)
    m, d = 21, 1160
    x0 = rand(torch, m, d, seed=5, dtype=dtype)
    dy0 = rand(torch, m, d, seed=6, dtype=dtype)
    w, b = rand(torch, d, seed=1, shift=1.0), rand(torch, d, seed=2)
    x, _ = strided(torch, x0, extra, offset)
    out, buf = strided(torch, torch.zeros_like(x0), extra, offset)
    y, mean, rstd = kq.layernorm(x, w, b, eps=EPS, out=out, stats=True)
    y0, mu, rs, y_tol, _, _ = ref.norm(x0, w, b, EPS)
    ref.assert_near(out, y0, y_tol, "y")
    assert int(buf.isnan().sum()) == buf.numel() - m * d
    dy, _ = strided(torch, dy0, extra, offset)
    dx, buf = strided(torch, torch.zeros_like(x0), extra, offset)
    _, dw, db = kq.layernorm_backward(dy, x, mean, rstd, w, dx=dx)
    want, tol = ref.norm_grad(dy0, x0, mean, rstd, w)
    for got, v, t, what in zip((dx, dw, db), want, tol, ("dx", "dw", "db")):
        ref.assert_near(got, v, t, what)
    assert int(buf.isnan().sum()) == buf.numel() - m * d


@pytest.mark.parametrize("dt", ["bfloat16", "float32"])
@pytest.mark.parametrize("m,d", SHAPES + [(16, 96), (17, 96), (9000, 72)])
def test_backward(torch, kq, m, d, dt):
    dtype = getattr(torch, dt)
    case("norm_grad %dx%d %s" % (m, d, dt))
    x = rand(torch, m, d, seed=m + d, scale=2.0, shift=0.5, dtype=dtype)
    dy = rand(torch, m, d, seed=m + d + 1, dtype=dtype)
    w = rand(torch, d, seed=1, shift=1.0)
    _, mean, rstd = kq.layernorm(x, w, None, eps=EPS, stats=True)
    for ww in (w, None):
        got = kq.layernorm_backward(dy, x, mean, rstd, ww)
        want, tol = ref.norm_grad(dy, x, mean, rstd, ww)
        for g, v, t, what in zip(got, want, tol, ("dx", "dw", "db")):
            ref.assert_near(g, v, t, what)
        again = kq.layernorm_backward(dy, x, mean, rstd, ww)
        assert all(torch.equal(a, b) for a, b in zip(got, again))  # a fixed order of sums
    dx, none, nothing = kq.layernorm_backward(dy, x, mean, rstd, None, params=False)
    assert torch.equal(dx, got[0]) and none is None and nothing is None


# widths for every number of waves and chunks that many rows take (whole rows and a partial last piece), and, at the
# end, calls of 128 MiB and more, whose accesses are non-temporal
MANY = [(260, 512), (300, 1000), (700, 1152), (260, 2048), (257, 2056), (512, 4096), (300, 4608), (290, 6144), (260, 8192),
        (258, 12288), (256, 16384), (33000, 1032), (8300, 4104), (5000, 8200), (2100, 16384)]


@pytest.mark.parametrize("dt", ["bfloat16", "float32"])
@pytest.mark.parametrize("m,d", MANY)
def test_many_rows(torch, kq, m, d, dt):
    dtype = getattr(torch, dt)
    case("norm, norm_grad %dx%d %s" % (m, d, dt))
    x = rand(torch, m, d, seed=m, scale=2.0, shift=0.5, dtype=dtype)
    dy = rand(torch, m, d, seed=d, dtype=dtype)
    w, b = rand(torch, d, seed=1, shift=1.0), rand(torch, d, seed=2)
    y, mean, rstd = kq.layernorm(x, w, b, eps=EPS, stats=True)
    y0, mu, rs, y_tol, mu_tol, rs_tol = ref.norm(x, w, b, EPS)
    ref.assert_near(y, y0, y_tol, "y")
    ref.assert_near(mean, mu, mu_tol, "mean")
    ref.assert_near(rstd, rs, rs * rs_tol, "rstd")
    del y, y0, y_tol
    got = kq.layernorm_backward(dy, x, mean, rstd, w)
    want, tol = ref.norm_grad(dy, x, mean, rstd, w)
    for g, v, t, what in zip(got, want, tol, ("dx", "dw", "db")):
        ref.assert_near(g, v, t, what)
    again = kq.layernorm_backward(dy, x, mean, rstd, w)
    assert all(torch.equal(a, b) for a, b in zip(got, again))


# the same number of pieces with widths that are no whole 16 bytes (a lane then takes every 64th element), and few rows
ODD = [(260, 511), (300, 999), (700, 1155), (260, 2047), (257, 2059), (512, 4093), (300, 4607), (290, 6145), (260, 8191),
       (258, 12289), (256, 16383), (33000, 1031), (8300, 4105), (5000, 8201), (2100, 16383), (9, 513), (5, 2051), (3, 9001),
       (4, 16381), (1, 16384 + 7)]


@pytest.mark.parametrize("dt", ["bfloat16", "float32"])
@pytest.mark.parametrize("m,d", ODD)
def test_odd_widths(torch, kq, m, d, dt):
    test_many_rows(torch, kq, m, d, dt)


@pytest.mark.parametrize("m", [5, 31, 33, 1025, 2100])
@pytest.mark.parametrize("d", [8, 500, 1001, 1152])
def test_backward_of_one_wave_rows(torch, kq, m, d):
    """Parts of fewer rows than waves, of some waves more than others; dweight and dbias each alone too."""
    case("norm_grad %dx%d" % (m, d))
    x, dy = rand(torch, m, d, seed=m, shift=0.5), rand(torch, m, d, seed=d)
    w = rand(torch, d, seed=1, shift=1.0)
    _, mean, rstd = kq.layernorm(x, w, eps=EPS, stats=True)
    got = kq.layernorm_backward(dy, x, mean, rstd, w)
    want, tol = ref.norm_grad(dy, x, mean, rstd, w)
    for g, v, t, what in zip(got, want, tol, ("dx", "dw", "db")):
        ref.assert_near(g, v, t, what)
    assert torch.equal(kq.layernorm_backward(dy, x, mean, rstd, w, params=False)[0], got[0])


def test_parameters_at_any_address(torch, kq):
    """weight, bias and their gradients 4-byte aligned only: the same values by the general path; the
    quantizing norm refuses them."""
    m, d = 40, 1024
    x = rand(torch, m, d, seed=1, dtype=torch.bfloat16)
    dy = rand(torch, m, d, seed=2, dtype=torch.bfloat16)
    buf = rand(torch, 4 * d + 8, seed=3, shift=1.0)
    w, b = buf[1:1 + d], buf[d + 2:2 * d + 2]
    y, mean, rstd = kq.layernorm(x, w, b, eps=EPS, stats=True)
    y0, mu, rs, y_tol, _, _ = ref.norm(x, w, b, EPS)
    ref.assert_near(y, y0, y_tol, "y")
    keep = buf.clone()
    dw, db = buf[2 * d + 3:3 * d + 3], buf[3 * d + 5:4 * d + 5]
    for rows in (m, 3):
        want, tol = ref.norm_grad(dy[:rows], x[:rows], mean[:rows], rstd[:rows], w)
        got = kq.layernorm_backward(dy[:rows], x[:rows], mean[:rows], rstd[:rows], w, dweight=dw, dbias=db)
        for g, v, t, what in zip(got, want, tol, ("dx", "dw", "db")):
            ref.assert_near(g, v, t, what)
    buf[2 * d + 3:3 * d + 3] = keep[2 * d + 3:3 * d + 3]
    buf[3 * d + 5:4 * d + 5] = keep[3 * d + 5:4 * d + 5]
    assert torch.equal(buf, keep)  # nothing beside them was written
    with pytest.raises(kq.KQError):
        kq.layernorm_quantize_mxfp4(x, w)


def test_large_offset_and_equal_rows(torch, kq):
    """A mean far from zero cancels without loss; a row of equal values gives the bias (x - mean is
    0 up to 2 u of the first mean's rounding, times rstd = 1 / sqrt(eps))."""
    for d in (24, 1000, 4096, 5000):
        x = rand(torch, 6, d, seed=d, shift=3000.0)
        b = rand(torch, d, seed=3)
        y, mean, rstd = kq.layernorm(x, None, b, eps=EPS, stats=True)
        y0, mu, rs, y_tol, mu_tol, rs_tol = ref.norm(x, None, b, EPS)
        ref.assert_near(y, y0, y_tol, "y")
        ref.assert_near(mean, mu, mu_tol, "mean")
        x = torch.full((3, d), 1000.1, device="cuda")
        y = kq.layernorm(x, None, b, eps=EPS)
        y0, mu, rs, y_tol, mu_tol, rs_tol = ref.norm(x, None, b, EPS)
        ref.assert_near(y, y0, y_tol, "equal")
        z = kq.layernorm(torch.zeros(2, d, device="cuda"), None, b, eps=EPS)
        assert torch.equal(z, b.expand(2, d))


def test_nan_and_infinity_stay_in_their_rows(torch, kq):
    for d in (100, 1024):
        x = rand(torch, 9, d, seed=1, dtype=torch.bfloat16)
        clean = kq.layernorm(x)
        x[2, 5] = float("nan")
        x[6, d - 1] = float("inf")
        y = kq.layernorm(x)
        assert bool(y[2].isnan().all()) and bool(y[6].isnan().all())
        keep = [0, 1, 3, 4, 5, 7, 8]
        assert torch.equal(y[keep], clean[keep])


@pytest.mark.parametrize("d", [40, 1030, 4096])
def test_statistics_of_rows_with_nan_and_infinity(torch, kq, d):
    """rstd is NaN too, so that the gradients of such a row are NaN and do not pass for numbers."""
    x = rand(torch, 8, d, seed=d)
    x[1, 3], x[4, d - 1], x[6, 0] = float("nan"), float("inf"), float("-inf")
    y, mean, rstd = kq.layernorm(x, eps=EPS, stats=True)
    bad = torch.zeros(8, dtype=torch.bool, device="cuda")
    bad[[1, 4, 6]] = True
    assert torch.equal(rstd.isnan(), bad) and torch.equal(mean.isfinite(), ~bad)
    assert torch.equal(y.isnan().all(1), bad) and torch.equal(y.isnan().any(1), bad)
    dx, _, _ = kq.layernorm_backward(rand(torch, 8, d, seed=2), x, mean, rstd)
    assert torch.equal(dx.isnan().all(1), bad) and torch.equal(dx.isnan().any(1), bad)


def test_no_rows(torch, kq):
    x = torch.empty(0, 48, device="cuda")
    w = torch.ones(48, device="cuda")
    y, mean, rstd = kq.layernorm(x, w, w, stats=True)
    assert y.shape == (0, 48) and mean.numel() == 0
    dw = torch.full((48,), 7.0, device="cuda")
    dx, dw, db = kq.layernorm_backward(x, x, mean, rstd, w, dweight=dw)
    assert dx.shape == (0, 48) and not bool(dw.any()) and not bool(db.any())
    codes, scales = kq.layernorm_quantize_mxfp4(torch.empty(0, 64, device="cuda"))
    assert codes.shape == (0, 32) and scales.shape == (0, 2)


def test_offsets_past_32_bits(torch, kq):
    """Rows whose element offsets pass 2^31 (a view of a 5 GiB buffer): the last ones are right."""
    ld, m, d = 1 << 20, 2500, 96
    buf = torch.empty(m * ld, dtype=torch.bfloat16, device="cuda")
    x = buf.view(m, ld)[:, 8:8 + d]
    x.copy_(rand(torch, m, d, seed=11, dtype=torch.bfloat16))
    w = rand(torch, d, seed=1, shift=1.0)
    y, mean, rstd = kq.layernorm(x, w, None, eps=EPS, stats=True)
    ref.assert_near(y, *[ref.norm(x, w, None, EPS)[i] for i in (0, 3)], "y")
    dy = rand(torch, m, d, seed=12, dtype=torch.bfloat16)
    out = buf.view(m, ld)[:, 4096:4096 + d]
    got = kq.layernorm_backward(dy, x, mean, rstd, w, dx=out)
    want, tol = ref.norm_grad(dy, x, mean, rstd, w)
    for g, v, t in zip(got, want, tol):
        ref.assert_near(g, v, t)
    xq = buf.view(m, ld)[:, 8:8 + d]
    c1, s1 = kq.layernorm_quantize_mxfp4(xq, w)
    c2, s2 = kq.layernorm_quantize_mxfp4(xq.contiguous(), w)
    assert torch.equal(c1, c2) and torch.equal(s1, s2)


# one block, widths that fill no wave, whole and partial segments of 512 channels, one to many waves
QSHAPES = [(1, 32), (3, 96), (70, 160), (5, 512), (33, 544), (19, 1152), (1, 4096), (40, 4608), (6, 8224), (3, 16384),
           (2, 32768), (300, 512), (257, 1056), (600, 1152), (260, 2048), (300, 4096), (258, 4608), (260, 5120), (256, 8192),
           (256, 12288), (257, 16384)]


@pytest.mark.parametrize("dt", ["bfloat16", "float32"])
@pytest.mark.parametrize("m,d", QSHAPES)
def test_quantize(torch, kq, m, d, dt):
    """In check mode y T is within its bound of 64 bits, and codes and scales are exactly the
    quantization of that y T; the mode changes neither, nor does the packed layout."""
    dtype = getattr(torch, dt)
    case("norm_quant %dx%d %s" % (m, d, dt))
    x = rand(torch, m, d, seed=m + d, scale=2.0, shift=0.5, dtype=dtype)
    w, b = rand(torch, d, seed=1, scale=0.3, shift=1.0), rand(torch, d, seed=2, scale=0.2)
    for kind in ("lu", "mixed", None):
        f = None if kind is None else (synth.lu_perturbed_factors(d // 32, 4) if kind == "lu" else
                                       synth.special_factors(d // 32, "mixed"))
        fac = None if f is None else torch.from_numpy(f).cuda()
        y = torch.empty((m, d), device="cuda")
        codes, scales, mean, rstd = kq.layernorm_quantize_mxfp4(x, w, b, fac, eps=EPS, y_debug=y, stats=True)
        c2, s2 = kq.layernorm_quantize_mxfp4(x, w, b, fac, eps=EPS)
        assert torch.equal(codes, c2) and torch.equal(scales, s2)
        parity.check_self_consistent(codes.cpu().numpy(), scales.cpu().numpy(), y.cpu().numpy())
        y0, mu, rs, y_tol, mu_tol, rs_tol = ref.norm(x, w, b, EPS)
        ref.assert_near(mean, mu, mu_tol, "mean")
        ref.assert_near(rstd, rs, rs * rs_tol, "rstd")
        yb, tb = y0.view(m, -1, 32), y_tol.view(m, -1, 32)
        if f is not None:
            k = np.ones((d // 32, 1, 1))
            for i in range(5):
                k = np.stack([np.kron(p, q) for p, q in zip(k, f[:, i].astype(np.float64))])
            k = torch.from_numpy(k).cuda()
            # per output channel, sum over r of |y_r K_rc|; each stage's mixing rounds by a few u
            # (the transform's own rule: 1e-5 of the block's norm), and the norm's bound passes through |K|
            want = torch.stack([yb[:, j] @ k[j] for j in range(d // 32)], 1)
            tol = torch.stack([tb[:, j] @ k[j].abs() for j in range(d // 32)], 1)
            tol = tol + 1e-5 * want.norm(dim=2, keepdim=True)
        else:
            want, tol = yb, tb
        ref.assert_near(y.view(m, -1, 32), want, tol, "y T")
        if d % 256 == 0:
            c3, p3 = kq.layernorm_quantize_mxfp4(x, w, b, fac, eps=EPS, packed=True)
            assert torch.equal(c3, codes) and torch.equal(p3.view(-1), kq.pack_mxfp4_scales(scales).view(-1))


def test_quantize_strided_and_plain_parameters(torch, kq):
    """Padded input rows; no weight and no bias."""
    x0 = rand(torch, 23, 1056, seed=9, dtype=torch.bfloat16)
    x, _ = strided(torch, x0, 24)
    a = kq.layernorm_quantize_mxfp4(x)
    b = kq.layernorm_quantize_mxfp4(x0, torch.ones(1056, device="cuda"), torch.zeros(1056, device="cuda"))
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_quantize_is_the_quantizer_of_the_norm(torch, kq):
    """With T = I the codes are those of quantize_mxfp4_f32 on the 32-bit norm."""
    x = rand(torch, 64, 2048, seed=4)
    w, b = rand(torch, 2048, seed=1, shift=1.0), rand(torch, 2048, seed=2)
    y = torch.empty(64, 2048, device="cuda")
    codes, scales = kq.layernorm_quantize_mxfp4(x, w, b, y_debug=y)
    c2, s2 = kq.quantize_mxfp4_f32(y)
    assert torch.equal(codes, c2) and torch.equal(scales, s2)


def test_refusals(torch, kq):
    x = torch.zeros(4, 64, device="cuda")
    v = torch.zeros(64, device="cuda")
    with pytest.raises(TypeError):
        kq.layernorm(x.half())
    with pytest.raises(TypeError):
        kq.layernorm(x, v.bfloat16())
    with pytest.raises(ValueError):
        kq.layernorm(x, v[:63])
    with pytest.raises(ValueError):
        kq.layernorm(x.t())
    with pytest.raises(ValueError):
        kq.layernorm(x[0])
    with pytest.raises(TypeError):
        kq.layernorm(x, out=x.bfloat16())
    with pytest.raises(ValueError):
        kq.layernorm(x, out=torch.zeros(4, 63, device="cuda"))
    with pytest.raises(kq.KQError):
        kq.layernorm(x, eps=-1.0)
    with pytest.raises(kq.KQError):
        kq.layernorm(x[:1].expand(4, 64))  # rows that overlap
    with pytest.raises(ValueError):
        kq.layernorm_backward(x, x, None, None)
    with pytest.raises(TypeError):
        kq.layernorm_backward(x.bfloat16(), x, v[:4], v[:4])
    with pytest.raises(ValueError):
        kq.layernorm_backward(x, x, v, v[:4])
    with pytest.raises(ValueError):
        kq.layernorm_backward(x, x, v[:4], v[:4], params=False, dbias=v)
    with pytest.raises(kq.KQError):
        kq.layernorm_backward(torch.zeros(40, 64, device="cuda"), torch.zeros(40, 64, device="cuda"),
                              torch.zeros(40, device="cuda"), torch.zeros(40, device="cuda"),
                              workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    with pytest.raises(kq.KQError):
        kq.layernorm_quantize_mxfp4(torch.zeros(2, 48, device="cuda"))
    with pytest.raises((ValueError, kq.KQError)):
        kq.layernorm_quantize_mxfp4(x, packed=True)
    with pytest.raises(ValueError):
        kq.layernorm_quantize_mxfp4(x, factors=v)


@pytest.mark.parametrize("dt", ["bfloat16", "float32"])
@pytest.mark.parametrize("m,d", [(3, 40), (300, 512), (300, 1152), (5, 4096), (300, 4096), (300, 4609), (260, 16384), (2, 20000)])
def test_mean_of_cancelling_values(torch, kq, m, d, dt):
    """The mean is summed in 64 bits whatever the type, the width and a lane's share of the row: large
    values that cancel, within eight neighbours and 64 apart, leave it with 64 bits' rounding. The
    sum of d terms is off by at most d 2^-53 of the sum of their magnitudes (its scaling by 1 / d adds 2
    such roundings) and the mean itself is rounded to fp32 once."""
    dtype = getattr(torch, dt)
    g = torch.Generator("cuda").manual_seed(d)
    x = torch.randn(m, d, generator=g, device="cuda")
    for apart in (1, 3, 64):
        at = torch.arange(0, max(0, d - apart), 2 * apart + 8, device="cuda")
        big = 1e4 * torch.rand(m, at.numel(), generator=g, device="cuda").to(dtype).float() + 256
        x[:, at], x[:, at + apart] = big, -big
    x = x.to(dtype)

    def near(mean):
        e = x.double()
        mu = e.mean(1)
        tol = ref.U * (1 + 2.0 ** -20) * mu.abs() + (d + 4) * 2.0 ** -53 * e.abs().mean(1)
        assert bool(((mean.double() - mu).abs() <= tol).all()), float(((mean.double() - mu).abs() / tol).max())

    near(kq.layernorm(x, eps=EPS, stats=True)[1])
    near(kq.layernorm(strided(torch, x, 3, 1)[0], eps=EPS, stats=True)[1])  # element by element
    if d % 32 == 0:
        near(kq.layernorm_quantize_mxfp4(x, eps=EPS, stats=True)[2])


def resident(torch, waves, per_cu):
    """Rows that the persistent grid has at a time with `per_cu` waves per compute unit."""
    return torch.cuda.get_device_properties(0).multi_processor_count * per_cu // waves


# a width for every shape that many rows take, whole rows and partial last pieces, with its waves per row and the most
# waves per compute unit that any of its launches keeps
LOOPED = [(512, 1, 16), (416, 1, 16), (1024, 1, 16), (1152, 1, 16), (2048, 2, 16), (4096, 4, 16), (2592, 4, 16), (4608, 3, 12),
          (5120, 4, 16), (8192, 8, 16), (12288, 8, 16), (16384, 8, 16), (14336, 8, 16)]


@pytest.mark.parametrize("dt", ["bfloat16", "float32"])
@pytest.mark.parametrize("d,waves,per_cu", LOOPED)
def test_rows_one_after_another(torch, kq, d, waves, per_cu, dt):
    """Three rows and more per workgroup or wave, and a remainder: the norm and the quantizing norm give each row
    what they give it in a call of as many rows as are resident at once, where no workgroup has a second one (the
    same shape of kernel, so the same bits); that call is checked against 64 bits by the other tests' bounds."""
    dtype = getattr(torch, dt)
    once = resident(torch, waves, 4)  # a row each whatever the launch keeps, and still the shapes of many rows
    once = max(once, torch.cuda.get_device_properties(0).multi_processor_count)
    m = 3 * resident(torch, waves, per_cu) + 5
    case("rows in turn %dx%d %s, %d at once" % (m, d, dt, once))
    x = rand(torch, m, d, seed=d, scale=2.0, shift=0.5, dtype=dtype)
    x *= torch.linspace(0.5, 3.0, m, device="cuda")[:, None].to(dtype)  # no two rows of one scale
    w, b = rand(torch, d, seed=1, scale=0.3, shift=1.0), rand(torch, d, seed=2, scale=0.2)
    fac = torch.from_numpy(synth.lu_perturbed_factors(d // 32, 4)).cuda()
    y, mean, rstd = kq.layernorm(x, w, b, eps=EPS, stats=True)
    quant = [kq.layernorm_quantize_mxfp4(x, w, b, f, eps=EPS, packed=p, stats=True)
             for f in (fac, None) for p in ((False, True) if d % 256 == 0 else (False,))]
    for lo in range(0, m, once):
        hi = min(m, lo + once)
        lo = max(0, hi - once)  # the last call has as many rows too
        rows = x[lo:hi]
        part = kq.layernorm(rows, w, b, eps=EPS, stats=True)
        assert all(torch.equal(a[lo:hi], c) for a, c in zip((y, mean, rstd), part)), (lo, hi)
        q = kq.layernorm_quantize_mxfp4(rows, w, b, fac, eps=EPS, stats=True)
        assert all(torch.equal(a[lo:hi], c) for a, c in zip(quant[0], q)), (lo, hi)
    y0, mu, rs, y_tol, mu_tol, rs_tol = ref.norm(x, w, b, EPS)
    ref.assert_near(y, y0, y_tol, "y")
    ref.assert_near(quant[0][2], mu, mu_tol, "mean")
    ref.assert_near(quant[0][3], rs, rs * rs_tol, "rstd")
    if d % 256 == 0:
        for plain, packed in ((quant[0], quant[1]), (quant[2], quant[3])):
            assert torch.equal(plain[0], packed[0]) and torch.equal(plain[2], packed[2]) and torch.equal(plain[3], packed[3])
            assert torch.equal(kq.pack_mxfp4_scales(plain[1]).view(-1), packed[1].view(-1))
    # T = I: the codes are those of the quantizer on the norm in check mode, row by row
    yt = torch.empty((m, d), device="cuda")
    plain = kq.layernorm_quantize_mxfp4(x, w, b, None, eps=EPS, y_debug=yt)
    want = kq.quantize_mxfp4_f32(yt)
    same = quant[-1] if d % 256 else quant[2]
    assert torch.equal(plain[0], want[0]) and torch.equal(plain[1], want[1])
    assert torch.equal(plain[0], same[0]) and torch.equal(plain[1], same[1])


@pytest.mark.parametrize("dt", ["bfloat16", "float32"])
@pytest.mark.parametrize("d,waves,per_cu", [(511, 1, 16), (999, 1, 16), (1155, 1, 16), (2047, 2, 16), (4093, 4, 16), (4607, 3, 12),
                                            (5123, 4, 16), (8191, 8, 16), (12281, 8, 16), (16383, 8, 16)])
def test_odd_rows_one_after_another(torch, kq, d, waves, per_cu, dt):
    """The same for the norm of rows that are no whole 16 bytes."""
    dtype = getattr(torch, dt)
    once = max(resident(torch, waves, 4), torch.cuda.get_device_properties(0).multi_processor_count)
    m = 3 * resident(torch, waves, per_cu) + 5
    x = rand(torch, m, d, seed=d, scale=2.0, shift=0.5, dtype=dtype)
    w, b = rand(torch, d, seed=1, scale=0.3, shift=1.0), rand(torch, d, seed=2, scale=0.2)
    got = kq.layernorm(x, w, b, eps=EPS, stats=True)
    for lo in range(0, m, once):
        hi = min(m, lo + once)
        lo = max(0, hi - once)
        part = kq.layernorm(x[lo:hi], w, b, eps=EPS, stats=True)
        assert all(torch.equal(a[lo:hi], c) for a, c in zip(got, part)), (lo, hi)
    y0, mu, rs, y_tol, mu_tol, rs_tol = ref.norm(x, w, b, EPS)
    ref.assert_near(got[0], y0, y_tol, "y")
    ref.assert_near(got[1], mu, mu_tol, "mean")
    ref.assert_near(got[2], rs, rs * rs_tol, "rstd")


def small_integers(torch, shape, seed, dtype):
    """-3 .. 3 without 0: a column's sum stays below 2^24 up to 2^22 rows, so that every order of fp32 sums is exact."""
    g = torch.Generator("cuda").manual_seed(seed)
    v = torch.randint(1, 4, shape, generator=g, device="cuda")
    return torch.where(torch.rand(shape, generator=g, device="cuda") < 0.5, -v, v).to(dtype)


# rows that leave remainders of the parts (at most 256, of 4 rows and more), of the rows that a workgroup has side by
# side (4 or 8) and of both; a width for every shape of the backward kernel, whole 16-byte rows and odd ones; at the end
# calls of 128 MiB and more, whose parts take every parts-th row
EXACT = [(m, d) for m in (1, 3, 5, 7, 9, 31, 33, 1023, 1025, 1027, 2053, 4111) for d in (8, 1000, 1001, 1152)] + \
    [(m, d) for m in (1, 6, 1025, 1531) for d in (513, 2048, 2047, 4096, 4093, 8192, 8191, 12288, 12281, 16384, 16383, 16400)] + \
    [(33001, 1032), (33001, 1031), (50021, 520), (11003, 4096), (11003, 4095), (5531, 8200), (2801, 16384), (2801, 16383)]


@pytest.mark.parametrize("dt", ["bfloat16", "float32"])
@pytest.mark.parametrize("m,d", EXACT)
def test_backward_sums_every_row_once(torch, kq, m, d, dt):
    """With dy small integers, x = 1 or -1, mean 0 and rstd 1 the parameters' gradients are integers without any
    rounding: a row left out or counted twice shows in every column."""
    dtype = getattr(torch, dt)
    dy = small_integers(torch, (m, d), m + d, dtype)
    x = torch.where(small_integers(torch, (m, d), m, torch.float32) > 0, 1.0, -1.0).to(dtype)
    zero, one = torch.zeros(m, device="cuda"), torch.ones(m, device="cuda")
    _, dw, db = kq.layernorm_backward(dy, x, zero, one)
    assert torch.equal(dw.double(), (dy.double() * x.double()).sum(0)), "dweight"
    assert torch.equal(db.double(), dy.double().sum(0)), "dbias"


@pytest.mark.parametrize("dt", ["bfloat16", "float32"])
@pytest.mark.parametrize("m,d", [(7, 1152), (300, 1152), (300, 4096), (5, 16400)])
def test_rows_at_unlike_addresses(torch, kq, m, d, dt):
    """Input, output and gradients each with a row stride and an address of its own, one of them not 16-byte aligned:
    within the bounds of the aligned call."""
    dtype = getattr(torch, dt)
    x0, dy0 = rand(torch, m, d, seed=5, dtype=dtype), rand(torch, m, d, seed=6, dtype=dtype)
    w, b = rand(torch, d, seed=1, shift=1.0), rand(torch, d, seed=2)
    y0, mu, rs, y_tol, mu_tol, rs_tol = ref.norm(x0, w, b, EPS)
    for odd in ("x", "y", "dy", "dx"):
        at = lambda name: (3, 1) if odd == name else (16, 0)
        x, _ = strided(torch, x0, *at("x"))
        dy, _ = strided(torch, dy0, *at("dy"))
        y, ybuf = strided(torch, torch.zeros_like(x0), *at("y"))
        dx, xbuf = strided(torch, torch.zeros_like(x0), *at("dx"))
        _, mean, rstd = kq.layernorm(x, w, b, eps=EPS, out=y, stats=True)
        ref.assert_near(y, y0, y_tol, odd)
        _, dw, db = kq.layernorm_backward(dy, x, mean, rstd, w, dx=dx)
        want, tol = ref.norm_grad(dy0, x0, mean, rstd, w)
        for got, v, t, what in zip((dx, dw, db), want, tol, ("dx", "dw", "db")):
            ref.assert_near(got, v, t, odd + " " + what)
        for buf in (ybuf, xbuf):
            assert int(buf.isnan().sum()) == buf.numel() - m * d


def test_more_wide_rows_than_workgroups(torch, kq):
    """Rows too wide for registers, more than the 65536 workgroups of their launch: the rows behind get what they get
    in a call of their own."""
    m, d, cut = 65536 + 700, 16416, 65536
    case("wide rows %dx%d" % (m, d))
    x = torch.empty(m, d, dtype=torch.bfloat16, device="cuda").normal_(generator=torch.Generator("cuda").manual_seed(3))
    w, b = rand(torch, d, seed=1, shift=1.0), rand(torch, d, seed=2)
    whole = kq.layernorm(x, w, b, eps=EPS, stats=True)
    part = kq.layernorm(x[cut:], w, b, eps=EPS, stats=True)
    assert all(torch.equal(a[cut:], c) for a, c in zip(whole, part))
    y, mean, rstd = whole
    y0, mu, rs, y_tol, _, _ = ref.norm(x[-600:], w, b, EPS)
    ref.assert_near(y[-600:], y0, y_tol, "y")
    codes, scales, _, _ = kq.layernorm_quantize_mxfp4(x, w, b, eps=EPS, stats=True)
    c2, s2 = kq.layernorm_quantize_mxfp4(x[cut:], w, b, eps=EPS)
    assert torch.equal(codes[cut:], c2) and torch.equal(scales[cut:], s2)
    dx = kq.layernorm_backward(y, x, mean, rstd, w, params=False)[0]
    want, tol = ref.norm_grad(y[-600:], x[-600:], mean[-600:], rstd[-600:], w)
    ref.assert_near(dx[-600:], want[0], tol[0], "dx")
