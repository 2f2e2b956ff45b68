"""GPU: both projections of a gated feed-forward block and their gate in one kernel (kq_mxfp4_gated_linear), and the
gradients of that epilogue, against 64-bit forms (tests/gated_ref.py)."""
import math

import pytest

from tests import gated_ref as ref
from tests import layer_ref

pytestmark = pytest.mark.gpu

ACTS = ["none", "relu", "silu", "gelu", "gelu_tanh"]


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


def check(torch, kq, m, n, k, name, dt, packed, bias=True, seed=0, pad=0):
    dtype = getattr(torch, dt)
    print("[case] gated %dx%dx%d %s %s packed=%d" % (m, n, k, name, dt, packed), flush=True)
    ca, sa = operand(torch, kq, m, k, seed + 1)
    (cg, sg), (cu, su) = (operand(torch, kq, n, k, seed + i, 1.0 if k == 0 else k ** -0.5) for i in (2, 3))
    bg, bu = (torch.randn(n, generator=gen(torch, seed + i), device="cuda") if bias else None for i in (4, 5))
    scales = [kq.pack_mxfp4_scales(s) if packed else s for s in (sa, sg, su)]
    args = (ca, scales[0], cg, scales[1], cu, scales[2])
    kw = dict(bias_g=bg, bias_u=bu, act=name, bf16=dt == "bfloat16", packed=packed)
    rooms = [torch.full((m, n + pad), math.nan, dtype=dtype, device="cuda") for _ in range(3)]
    out, g, u = kq.mxfp4_gated_linear(*args, out=rooms[0][:, :n], g=rooms[1][:, :n], u=rooms[2][:, :n], **kw)
    o64, g64, u64, o_tol, g_tol, u_tol = ref.forward(ca, sa, cg, sg, cu, su, bg, bu, name, dtype)
    layer_ref.assert_near(g, g64, g_tol, "g")
    layer_ref.assert_near(u, u64, u_tol, "u")
    layer_ref.assert_near(out, o64, o_tol, "out")
    for r in rooms:
        assert int(r.isnan().sum()) == m * pad  # the padding is left alone
    alone = kq.mxfp4_gated_linear(*args, **kw)
    assert torch.equal(alone, out)  # g and u asked for or not, padded or not, twice: the same output


# one token, a few, one past and one short of a tile; k of one block, of part of a stage, of many; odd n
SMALL = [(1, 16, 32), (1, 1, 64), (2, 33, 96), (7, 100, 1152), (16, 256, 512), (17, 130, 4096), (1, 1000, 2080),
         (33, 515, 288), (45, 1000, 1152), (64, 64, 2048), (65, 257, 640), (130, 300, 1056), (250, 129, 4608),
         (1, 8192, 256), (3, 5, 8192), (1, 11008, 4096), (31, 2001, 512), (32, 4000, 2304)]


@pytest.mark.parametrize("dt", ["bfloat16", "float32"])
@pytest.mark.parametrize("m,n,k", SMALL)
def test_few_rows(torch, kq, m, n, k, dt):
    for packed in [False, True] if k % 256 == 0 else [False]:
        check(torch, kq, m, n, k, ACTS[(m + n) % 5], dt, packed, seed=m)
        check(torch, kq, m, n, k, ACTS[(m + n + 1) % 5], dt, packed, bias=False, seed=n, pad=3)


# whole and ragged tiles of every kernel of more rows, k of whole stages, of half ones, of single blocks
LARGE = [(256, 256, 256), (1024, 2048, 512), (700, 650, 1152), (2048, 1024, 384), (1111, 1111, 768), (3000, 2052, 128),
         (513, 4095, 256), (4096, 260, 1056), (5000, 512, 96), (100, 2050, 2080), (130, 2046, 4096), (200, 2046, 1152),
         (600, 2049, 1024), (2050, 577, 2304), (2050, 578, 2336), (1500, 1666, 4096), (1500, 1668, 3968),
         (2048, 4096, 1152), (4000, 5000, 1024), (2000, 3001, 256), (400, 8200, 512), (60, 7000, 1024), (90, 1, 256),
         (65, 2017, 32), (129, 2017, 1056), (257, 2017, 288), (1537, 1281, 96), (1537, 1281, 1280), (257, 129, 512)]


@pytest.mark.parametrize("m,n,k", LARGE)
def test_many_rows(torch, kq, m, n, k):
    for i, packed in enumerate([False, True] if k % 256 == 0 else [False]):
        for j, dt in enumerate(("bfloat16", "float32")):
            check(torch, kq, m, n, k, ACTS[(m + k // 32 + i + j) % 5], dt, packed, bias=j == 0, seed=m, pad=(0, 8, 5)[(m + j) % 3])


# the 256 x 128 kernel: one tile per workgroup and several, whole ones and halves, and a workgroup that goes from one kind
# to the other; two stages of k, odd and even numbers of them, a partial one
BIG = [(4000, 5000, 1024), (4100, 5501, 512), (4097, 11001, 768), (2048, 5504, 2048), (5000, 8193, 1280), (1024, 5504, 4096),
       (2500, 6401, 1152), (8192, 2752, 896), (1030, 11008, 2304), (1000, 2751, 2048), (768, 4096, 4096), (2500, 7000, 1920), (4096, 4224, 512)]


@pytest.mark.parametrize("m,n,k", BIG)
def test_large_tiles(torch, kq, m, n, k):
    for i, packed in enumerate([False, True] if k % 256 == 0 else [False]):
        for j, dt in enumerate(("bfloat16", "float32")):
            check(torch, kq, m, n, k, ACTS[(m // 100 + k // 128 + 2 * i + j) % 5], dt, packed, bias=(i + j) % 2 == 0, seed=n,
                  pad=8 * (n % 8 == 0))


@pytest.mark.parametrize("name", ACTS)
@pytest.mark.parametrize("dt", ["bfloat16", "float32"])
def test_activations(torch, kq, name, dt):
    """Every activation over a wide range of g (the bias spreads it), on kernels for few and for many rows."""
    for m, n, k in ((5, 1024, 256), (300, 1024, 256), (2100, 1024, 256), (4096, 4096, 512)):
        ops = [operand(torch, kq, r, k, i, s) for i, (r, s) in enumerate(((m, 1.0), (n, k ** -0.5), (n, k ** -0.5)))]
        bg = torch.linspace(-12, 12, n, device="cuda")
        flat = [t for o in ops for t in o]
        out, g, u = kq.mxfp4_gated_linear(*flat, bias_g=bg, act=name, bf16=dt == "bfloat16", want_pre=True)
        o64, g64, u64, o_tol, g_tol, u_tol = ref.forward(*flat, bg, None, name, out.dtype)
        layer_ref.assert_near(g, g64, g_tol, "g")
        layer_ref.assert_near(u, u64, u_tol, "u")
        layer_ref.assert_near(out, o64, o_tol, "out")


@pytest.mark.parametrize("m,n", [(5, 40), (40, 72), (200, 4100), (1030, 4000)])
def test_no_inner_dimension(torch, kq, m, n):
    for packed in (False, True):
        check(torch, kq, m, n, 0, "silu", "float32", packed)
        check(torch, kq, m, n, 0, "gelu", "bfloat16", packed, bias=False)


def test_empty(torch, kq):
    for m, n in ((0, 8), (8, 0), (0, 0)):
        ops = [t for i, r in enumerate((m, n, n)) for t in operand(torch, kq, r, 64, i)]
        assert kq.mxfp4_gated_linear(*ops).shape == (m, n)
        dout = torch.empty(m, n, device="cuda")
        dg, du, bg, bu = kq.mxfp4_gated_linear_backward(dout, dout, dout)
        assert dg.shape == du.shape == (m, n) and bool((bg == 0).all()) and bool((bu == 0).all()) and bg.numel() == n


@pytest.mark.parametrize("m,n,k", [(9, 300, 512), (25, 300, 512), (60, 1901, 2304), (600, 2049, 1024), (2050, 577, 2304)])
def test_scales_at_any_address(torch, kq, m, n, k):
    """MX-layout scales need no alignment, each operand's its own: at odd addresses, the same values."""
    (ca, sa), (cg, sg), (cu, su) = (operand(torch, kq, r, k, i, s) for i, (r, s) in
                                    enumerate(((m, 1.0), (n, k ** -0.5), (n, k ** -0.5))))

    def moved(s, by):
        buf = torch.empty(s.numel() + by, dtype=torch.uint8, device="cuda")
        v = buf[by:].view(s.shape)
        v.copy_(s)
        return v

    o64, _, _, o_tol, _, _ = ref.forward(ca, sa, cg, sg, cu, su, None, None, "relu", torch.float32)
    for by in ((0, 0, 0), (1, 3, 2), (0, 1, 0), (0, 0, 1), (4, 4, 4), (0, 0, 4)):
        got = kq.mxfp4_gated_linear(ca, moved(sa, by[0]), cg, moved(sg, by[1]), cu, moved(su, by[2]), act="relu", bf16=False)
        layer_ref.assert_near(got, o64, o_tol, str(by))


@pytest.mark.parametrize("m,n,k", [(9, 301, 512), (300, 2049, 1024), (2050, 1155, 2304)])
def test_packed_scales_8_bytes_aligned(torch, kq, m, n, k):
    ops = [operand(torch, kq, r, k, i, s) for i, (r, s) in enumerate(((m, 1.0), (n, k ** -0.5), (n, k ** -0.5)))]
    packed = [kq.pack_mxfp4_scales(s) for _, s in ops]
    want = kq.mxfp4_gated_linear(ops[0][0], packed[0], ops[1][0], packed[1], ops[2][0], packed[2], packed=True, bf16=False)
    flat = [t for o in ops for t in o]
    o64, _, _, o_tol, _, _ = ref.forward(*flat, None, None, "silu", torch.float32)
    layer_ref.assert_near(want, o64, o_tol)
    for i in range(3):
        moved = list(packed)
        buf = torch.empty(packed[i].numel() + 8, dtype=torch.uint8, device="cuda")
        moved[i] = buf[8:].view(packed[i].shape)
        moved[i].copy_(packed[i])
        got = kq.mxfp4_gated_linear(ops[0][0], moved[0], ops[1][0], moved[1], ops[2][0], moved[2], packed=True, bf16=False)
        layer_ref.assert_near(got, o64, o_tol)


@pytest.mark.parametrize("m,n", [(3, 40), (40, 2040), (300, 2000), (2048, 2048)])
def test_halves_of_one_weight(torch, kq, m, n):
    """The two weights as halves of a fused one; the outputs as columns of one tensor and at odd addresses."""
    k = 512
    ca, sa = operand(torch, kq, m, k, 1)
    cw, sw = operand(torch, kq, 2 * n, k, 2, k ** -0.5)
    want = kq.mxfp4_gated_linear(ca, sa, cw[:n].clone(), sw[:n].clone(), cw[n:].clone(), sw[n:].clone(), want_pre=True)
    both = torch.full((m, 2 * n + 3), math.nan, dtype=torch.bfloat16, device="cuda")
    got = kq.mxfp4_gated_linear(ca, sa, cw[:n], sw[:n], cw[n:], sw[n:], g=both[:, 1:n + 1], u=both[:, n + 2:2 * n + 2])
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert bool(both[:, [0, n + 1, 2 * n + 2]].isnan().all())
    # one product of the whole weight has the same sums, up to its own kernel's order
    z = kq.mxfp4_linear(ca, sa, cw, sw, bf16=False)
    _, g64, u64, _, g_tol, u_tol = ref.forward(ca, sa, cw[:n], sw[:n], cw[n:], sw[n:], None, None, "silu", torch.float32)
    layer_ref.assert_near(z, torch.cat((g64, u64), 1), torch.cat((g_tol, u_tol), 1))


GRADS = [(1, 1), (1, 4096), (7, 100), (33, 513), (301, 4607), (500, 512), (64, 8192), (1000, 4001), (1030, 2048), (4096, 24),
         (5, 11008), (2, 70000), (384, 1000), (385, 1000), (384, 517), (129, 24)]


@pytest.mark.parametrize("dt", ["bfloat16", "float32"])
@pytest.mark.parametrize("m,n", GRADS)
def test_gradients(torch, kq, m, n, dt):
    dtype = getattr(torch, dt)
    for i, name in enumerate(ACTS):
        pad = (0, 8, 3)[(m + i) % 3]
        dout, g, u = (torch.full((m, n + pad), math.nan, dtype=dtype, device="cuda")[:, :n] for _ in range(3))
        for j, (t, s) in enumerate(((dout, 1.0), (g, 2.0), (u, 1.0))):
            t.copy_(torch.randn(m, n, generator=gen(torch, m + 10 * j), device="cuda") * s)
        rooms = [torch.full((m, n + pad), math.nan, dtype=dtype, device="cuda") for _ in range(2)]
        got = kq.mxfp4_gated_linear_backward(dout, g, u, act=name, dg=rooms[0][:, :n], du=rooms[1][:, :n])
        want, tol = ref.backward(dout, g, u, name)
        for what, a, b, t in zip(("dg", "du", "dbias_g", "dbias_u"), got, want, tol):
            layer_ref.assert_near(a, b, t, name + " " + what)
        assert all(int(r.isnan().sum()) == m * pad for r in rooms)
        again = kq.mxfp4_gated_linear_backward(dout, g, u, act=name)
        assert all(torch.equal(a, b) for a, b in zip(got, again))
        alone = kq.mxfp4_gated_linear_backward(dout, g, u, act=name, biases=False)
        assert torch.equal(alone[0], got[0]) and torch.equal(alone[1], got[1]) and alone[2] is None and alone[3] is None


def test_gradients_in_place_and_halves(torch, kq):
    m, n = 130, 1000
    dout, g, u = (torch.randn(m, n, generator=gen(torch, i), device="cuda").to(torch.bfloat16) for i in range(3))
    want = kq.mxfp4_gated_linear_backward(dout, g, u)
    both = torch.empty(m, 2 * n, dtype=torch.bfloat16, device="cuda")
    got = kq.mxfp4_gated_linear_backward(dout, g, u, dg=both[:, :n], du=both[:, n:])
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    g2, u2 = g.clone(), u.clone()
    got = kq.mxfp4_gated_linear_backward(dout, g2, u2, dg=g2, du=u2)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    d2, u2 = dout.clone(), u.clone()
    got = kq.mxfp4_gated_linear_backward(d2, g, u2, dg=d2, du=u2)
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_gradients_of_very_many_columns(torch, kq):
    """More columns than a launch has strips for: few rows, taken by rows."""
    n = (1 << 27) + 24
    dout, g, u = (torch.randn(2, n, generator=gen(torch, i), device="cuda").to(torch.bfloat16) for i in range(3))
    got = kq.mxfp4_gated_linear_backward(dout, g, u)
    for at in (slice(0, 3000), slice(n // 2 - 7, n // 2 + 3000), slice(n - 3000, n)):
        want, tol = ref.backward(dout[:, at], g[:, at], u[:, at], "silu")
        for what, a, b, t in zip(("dg", "du", "dbias_g", "dbias_u"), got, want, tol):
            layer_ref.assert_near(a[..., at], b, t, what)


def test_summed_gradients_of_integers(torch, kq):
    """Every row counts once in either sum: integers, exact in fp32."""
    for m, n in ((1, 40), (3, 513), (37, 24), (300, 1000), (384, 40), (384, 33), (385, 40), (1025, 520), (5000, 9)):
        for dt in (torch.bfloat16, torch.float32):
            dout, g, u = (torch.randint(-3, 4, (m, n), generator=gen(torch, m + i), device="cuda").to(dt) for i in range(3))
            dg, du, bg, bu = kq.mxfp4_gated_linear_backward(dout, g, u, act="none")
            d, gg, uu = dout.double(), g.double(), u.double()
            assert torch.equal(bg.double(), (d * uu).sum(0)) and torch.equal(bu.double(), (d * gg).sum(0))
            assert torch.equal(dg.double(), d * uu) and torch.equal(du.double(), d * gg)


def test_each_sum_alone(torch, kq):
    """Through the C entry point: a NULL output is left out, the others' bits stay."""
    m, n = 50, 600
    dout, g, u = (torch.randn(m, n, generator=gen(torch, i), device="cuda") for i in range(3))
    want = kq.mxfp4_gated_linear_backward(dout, g, u, act="gelu")
    ws = torch.empty(1 << 20, dtype=torch.uint8, device="cuda")
    for which in range(4):
        out = [torch.empty(m, n, device="cuda") if i < 2 else torch.empty(n, device="cuda") for i in range(4)]
        p = [t.data_ptr() if i == which else None for i, t in enumerate(out)]
        kq._check("kq_mxfp4_gated_linear_backward", kq.lib().kq_mxfp4_gated_linear_backward(
            dout.data_ptr(), n, g.data_ptr(), n, u.data_ptr(), n, 0, m, n, 3, p[0], n, p[1], n, p[2], p[3], ws.data_ptr(),
            ws.numel(), torch.cuda.current_stream().cuda_stream))
        assert torch.equal(out[which], want[which])


def test_gradient_against_differences(torch, kq):
    """The kernel's gradient along a direction, and a central difference of the 64-bit form: off by e^2 / 6 times the
    third derivative (at most 10 |v|^3 (1 + |u|) here) and 2^-50 of the loss over e."""
    m, n, e = 9, 200, 1e-4
    dout, g, u = (torch.randn(m, n, generator=gen(torch, i), device="cuda") for i in range(3))
    for name in ("none", "silu", "gelu", "gelu_tanh"):
        got = kq.mxfp4_gated_linear_backward(dout, g, u, act=name)
        _, tol = ref.backward(dout, g, u, name)
        for i, v in enumerate(torch.randn(2, m, n, generator=gen(torch, 7), device="cuda", dtype=torch.float64)):
            def loss(s):
                gg, uu = g.double() + (s * e * v if i == 0 else 0), u.double() + (s * e * v if i == 1 else 0)
                return (layer_ref.act(gg, name)[0] * uu * dout.double()).sum()
            diff = (loss(1) - loss(-1)) / (2 * e)
            mag = dout.abs().double()
            slack = ((tol[i] + layer_ref.half_step(torch.float32, got[i].double())) * v.abs()).sum() + \
                e * e / 6 * 10 * (mag * v.abs() ** 3 * (1 + u.abs())).sum() + 2.0 ** -50 * (mag * (g * u).abs()).sum() / e
            assert abs(float(diff - (got[i].double() * v).sum())) <= float(slack), name


def test_streams_and_graphs(torch, kq):
    for m, n, k in ((3, 520, 512), (40, 520, 512), (300, 2000, 512), (1000, 2048, 512)):
        ops = [t for i, (r, s) in enumerate(((m, 1.0), (n, k ** -0.5), (n, k ** -0.5))) for t in operand(torch, kq, r, k, i, s)]
        dout = torch.randn(m, n, device="cuda").to(torch.bfloat16)

        def step(stream=None):
            out, g, u = kq.mxfp4_gated_linear(*ops, want_pre=True, stream=stream)
            return (out, g, u, *kq.mxfp4_gated_linear_backward(dout, g, u, stream=stream))

        want = step()
        torch.cuda.synchronize()
        streams = [torch.cuda.Stream() for _ in range(2)]
        got = [step(s) for _ in range(3) for s in streams]
        torch.cuda.synchronize()
        for o in got:
            assert all(torch.equal(a, b) for a, b in zip(o, want))
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = step()
        for i in range(3):
            c, s = operand(torch, kq, m, k, 50 + i)
            ops[0].copy_(c)
            ops[1].copy_(s)
            graph.replay()
            torch.cuda.synchronize()
            want = step()
            assert all(torch.equal(a, b) for a, b in zip(out, want))


def test_outputs_past_32_bits(torch, kq):
    """More than 2^31 elements of the output: the last rows and columns."""
    m, n, k = 70000, 31000, 32
    ca, sa = operand(torch, kq, m, k, 1)
    cg, sg = operand(torch, kq, n, k, 2)
    cu, su = operand(torch, kq, n, k, 3)
    out = kq.mxfp4_gated_linear(ca, sa, cg, sg, cu, su)
    o64, _, _, tol, _, _ = ref.forward(ca[-300:], sa[-300:], cg, sg, cu, su, None, None, "silu", torch.bfloat16)
    layer_ref.assert_near(out[-300:], o64, tol)


def test_refusals_of_the_binding(torch, kq):
    ops = [t for i, r in enumerate((4, 8, 8)) for t in operand(torch, kq, r, 64, i)]
    names = ("codes_a", "scales_a", "codes_g", "scales_g", "codes_u", "scales_u")
    good = dict(zip(names, ops))
    for kw, error in [(dict(codes_a=ops[0].int()), TypeError), (dict(codes_a=ops[0].cpu()), TypeError),
                      (dict(codes_u=ops[4][:7]), ValueError), (dict(codes_g=ops[2][:, :16].contiguous()), ValueError),
                      (dict(scales_u=ops[5][:, :1]), ValueError), (dict(scales_g=ops[3].cpu()), TypeError), (dict(act="tanh"), ValueError),
                      (dict(bias_g=torch.zeros(7, device="cuda")), ValueError), (dict(bias_u=torch.zeros(8)), ValueError),
                      (dict(packed=True), kq.KQError), (dict(g=torch.zeros(4, 8, device="cuda")), TypeError),
                      (dict(u=torch.zeros(4, 9, dtype=torch.bfloat16, device="cuda")), ValueError),
                      (dict(out=torch.zeros(8, 4, dtype=torch.bfloat16, device="cuda").t()), ValueError)]:
        with pytest.raises(error):
            kq.mxfp4_gated_linear(**{**good, **kw})
    d = torch.zeros(4, 8, device="cuda")
    for kw, error in [(dict(g=d.bfloat16()), TypeError), (dict(u=d[:3]), ValueError), (dict(dout=d.half()), TypeError),
                      (dict(act="x"), ValueError), (dict(dbias_g=torch.zeros(9, device="cuda")), ValueError),
                      (dict(biases=False, dbias_u=torch.zeros(8, device="cuda")), ValueError),
                      (dict(dg=torch.zeros(1, 8, device="cuda").expand(4, 8)), kq.KQError)]:
        with pytest.raises(error):
            kq.mxfp4_gated_linear_backward(**{"dout": d, "g": d, "u": d, **kw})
    d = torch.zeros(400, 8, device="cuda")
    with pytest.raises(kq.KQError):
        kq.mxfp4_gated_linear_backward(d, d, d, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
