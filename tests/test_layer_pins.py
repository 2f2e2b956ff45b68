"""CPU: the 64-bit forms of tests/layer_ref.py against differences and torch's own functions, and the
refusals of the entry points around the W4A4 product (checked on the host before any HIP call)."""
import ctypes

import pytest
import torch

import mxfp4_activation_quantizer_amd as kq
from tests import layer_ref as ref

P = ctypes.c_void_p
GOOD = P(0x10000)  # never dereferenced: every case below fails or returns before a launch
ODD = P(0x10002)
BIG = 1 << 31


def slope_of(f, x, step=1e-6):
    """Central differences of the scalar f at every element of x."""
    g = torch.empty_like(x)
    flat, out = x.view(-1), g.view(-1)
    for i in range(flat.numel()):
        keep = float(flat[i])
        flat[i] = keep + step
        a = float(f())
        flat[i] = keep - step
        b = float(f())
        flat[i] = keep
        out[i] = (a - b) / (2 * step)
    return g


def test_norm_matches_torch():
    g = torch.Generator().manual_seed(1)
    x = torch.randn(5, 37, generator=g, dtype=torch.float64) * 3 + 2
    w, b = torch.randn(37, generator=g, dtype=torch.float64), torch.randn(37, generator=g, dtype=torch.float64)
    y = ref.norm(x, w, b, 1e-5)[0]
    assert torch.allclose(y, torch.nn.functional.layer_norm(x, (37,), w, b, 1e-5), atol=1e-12)


def test_norm_gradient_matches_differences():
    g = torch.Generator().manual_seed(2)
    x = torch.randn(4, 9, generator=g, dtype=torch.float64) + 0.5
    w, b = torch.randn(9, generator=g, dtype=torch.float64), torch.randn(9, generator=g, dtype=torch.float64)
    dy = torch.randn(4, 9, generator=g, dtype=torch.float64)

    def loss():
        return (ref.norm(x, w, b, 1e-3)[0] * dy).sum()

    _, mean, rstd = ref.norm(x, w, b, 1e-3)[:3]
    (dx, dw, db), _ = ref.norm_grad(dy, x, mean, rstd, w)
    # differences of step 1e-6 in 64 bits: 1e-12 of the third derivative, 1e-10 of rounding
    for got, leaf in ((dx, x), (dw, w), (db, b)):
        assert torch.allclose(got, slope_of(loss, leaf), atol=1e-7)


@pytest.mark.parametrize("name", list(kq.ACTS))
def test_activation_matches_torch_and_differences(name):
    z = torch.linspace(-9, 9, 181, dtype=torch.float64) + 0.013
    f = torch.nn.functional
    want = {"none": z, "relu": f.relu(z), "silu": f.silu(z), "gelu": f.gelu(z),
            "gelu_tanh": f.gelu(z, approximate="tanh")}[name]
    v, s = ref.act(z, name)
    assert torch.allclose(v, want, atol=1e-12)
    h = 1e-6
    assert torch.allclose(s, (ref.act(z + h, name)[0] - ref.act(z - h, name)[0]) / (2 * h), atol=1e-7)


def test_linear_gradient_matches_differences():
    g = torch.Generator().manual_seed(3)
    z = torch.randn(3, 5, generator=g, dtype=torch.float64)
    bias = torch.randn(5, generator=g, dtype=torch.float64)
    dout = torch.randn(3, 5, generator=g, dtype=torch.float64)
    (dz, dbias), _ = ref.linear_grad(dout, z + bias, "silu")
    assert torch.allclose(dz, slope_of(lambda: (ref.act(z + bias, "silu")[0] * dout).sum(), z), atol=1e-7)
    assert torch.allclose(dbias, slope_of(lambda: (ref.act(z + bias, "silu")[0] * dout).sum(), bias), atol=1e-7)


@pytest.fixture(scope="module")
def lib():
    return kq.lib()


def norm_args(**k):
    a = dict(X=GOOD, type=1, m=4, d=64, ldx=64, w=GOOD, b=GOOD, eps=1e-5, Y=GOOD, ldy=64, mean=GOOD, rstd=GOOD)
    a.update(k)
    return (*a.values(), None)


def grad_args(**k):
    a = dict(dY=GOOD, lddy=64, X=GOOD, ldx=64, type=1, m=64, d=64, w=GOOD, mean=GOOD, rstd=GOOD, dX=GOOD, lddx=64,
             dw=GOOD, db=GOOD, ws=GOOD, bytes=1 << 20)
    a.update(k)
    return (*a.values(), None)


def quant_args(**k):
    a = dict(X=GOOD, type=1, m=4, d=256, ldx=256, w=GOOD, b=GOOD, eps=1e-5, f=GOOD, codes=GOOD, scales=GOOD, packed=0,
             y=None, mean=GOOD, rstd=GOOD)
    a.update(k)
    return (*a.values(), None)


def linear_args(**k):
    a = dict(ca=GOOD, sa=GOOD, cw=GOOD, sw=GOOD, packed=0, m=4, n=8, k=64, bias=GOOD, act=0, type=1, res=GOOD, ldr=8,
             O=GOOD, ldo=8, Z=GOOD, ldz=8)
    a.update(k)
    return (*a.values(), None)


def lgrad_args(**k):
    a = dict(dO=GOOD, lddo=8, Z=GOOD, ldz=8, type=1, m=64, n=8, act=2, dZ=GOOD, lddz=8, db=GOOD, ws=GOOD,
             bytes=1 << 20)
    a.update(k)
    return (*a.values(), None)


SHAPE, NULL, ALIGN, UNSUP, OK = kq.KQ_ERR_SHAPE, kq.KQ_ERR_NULL, kq.KQ_ERR_ALIGN, kq.KQ_ERR_UNSUPPORTED, kq.KQ_OK
INF, NAN = float("inf"), float("nan")


@pytest.mark.parametrize("fn,make,change,status", [
    *[("kq_layernorm", norm_args, c, s) for c, s in [
        (dict(m=-1), SHAPE), (dict(d=-1), SHAPE), (dict(ldx=63), SHAPE), (dict(ldy=63), SHAPE),
        (dict(eps=-1e-9), SHAPE), (dict(eps=INF), SHAPE), (dict(eps=NAN), SHAPE), (dict(type=2), UNSUP),
        (dict(type=-1), UNSUP), (dict(m=BIG), UNSUP), (dict(ldx=BIG), UNSUP), (dict(ldy=BIG), UNSUP),
        (dict(X=None), NULL), (dict(Y=None), NULL), (dict(X=P(0x10001)), ALIGN), (dict(Y=P(0x10001)), ALIGN),
        (dict(X=ODD, type=0), ALIGN), (dict(w=ODD), ALIGN), (dict(b=ODD), ALIGN), (dict(mean=ODD), ALIGN),
        (dict(rstd=ODD), ALIGN), (dict(m=0, X=None, Y=None), OK), (dict(d=0, X=None, Y=None), OK)]],
    *[("kq_layernorm_backward", grad_args, c, s) for c, s in [
        (dict(m=-1), SHAPE), (dict(lddy=63), SHAPE), (dict(ldx=63), SHAPE), (dict(lddx=63), SHAPE),
        (dict(type=3), UNSUP), (dict(lddx=BIG), UNSUP), (dict(dY=None), NULL), (dict(X=None), NULL),
        (dict(mean=None), NULL), (dict(rstd=None), NULL), (dict(dX=None), NULL), (dict(ws=None), NULL),
        (dict(ws=P(0x10008)), ALIGN), (dict(bytes=4 * 2 * 64 * 4 - 1), SHAPE), (dict(dX=ODD, type=0), ALIGN),
        (dict(dw=ODD), ALIGN), (dict(db=ODD), ALIGN), (dict(w=ODD), ALIGN), (dict(mean=ODD), ALIGN),
        (dict(m=0, dw=None, db=None, dY=None, X=None, dX=None), OK), (dict(d=0, dY=None), OK)]],
    *[("kq_layernorm_quantize_mxfp4", quant_args, c, s) for c, s in [
        (dict(m=-1), SHAPE), (dict(d=48, ldx=48), SHAPE), (dict(d=64, ldx=64, packed=1), SHAPE), (dict(ldx=248), SHAPE),
        (dict(eps=-1.0), SHAPE), (dict(type=7), UNSUP), (dict(d=32800, ldx=32800), UNSUP),
        (dict(m=1 << 30, packed=1), UNSUP), (dict(m=BIG), UNSUP), (dict(X=None), NULL), (dict(codes=None), NULL),
        (dict(scales=None), NULL), (dict(X=P(0x10008)), ALIGN), (dict(ldx=260), ALIGN), (dict(type=0, ldx=258), ALIGN),
        (dict(codes=P(0x10004)), ALIGN), (dict(w=P(0x10004)), ALIGN), (dict(b=P(0x10004)), ALIGN),
        (dict(f=P(0x10004)), ALIGN), (dict(y=P(0x10004)), ALIGN), (dict(mean=ODD), ALIGN), (dict(rstd=ODD), ALIGN),
        (dict(m=0, X=None, codes=None, scales=None), OK)]],
    *[("kq_mxfp4_linear", linear_args, c, s) for c, s in [
        (dict(k=48), SHAPE), (dict(k=-32), SHAPE), (dict(m=-1), SHAPE), (dict(packed=1), SHAPE), (dict(ldo=7), SHAPE),
        (dict(ldr=7), SHAPE), (dict(ldz=7), SHAPE), (dict(act=5), UNSUP), (dict(act=-1), UNSUP), (dict(type=2), UNSUP),
        (dict(k=1 << 24), UNSUP), (dict(ldo=1 << 24), UNSUP), (dict(ldr=1 << 24), UNSUP), (dict(ldz=1 << 24), UNSUP),
        (dict(m=1 << 30), UNSUP), (dict(n=1 << 30, ldo=1 << 30, ldr=1 << 30, ldz=1 << 30), UNSUP), (dict(ca=None), NULL),
        (dict(sa=None), NULL), (dict(cw=None), NULL), (dict(sw=None), NULL), (dict(O=None), NULL),
        (dict(ca=P(0x10008)), ALIGN), (dict(cw=P(0x10008)), ALIGN), (dict(packed=1, k=256, sa=P(0x10004)), ALIGN),
        (dict(packed=1, k=256, sw=P(0x10004)), ALIGN), (dict(bias=ODD), ALIGN), (dict(O=P(0x10001)), ALIGN),
        (dict(res=P(0x10001)), ALIGN), (dict(Z=P(0x10001)), ALIGN), (dict(O=ODD, type=0), ALIGN),
        (dict(m=0, ca=None, O=None), OK), (dict(n=0, cw=None, O=None, ldo=0, ldr=0, ldz=0), OK)]],
    *[("kq_mxfp4_linear_backward", lgrad_args, c, s) for c, s in [
        (dict(m=-1), SHAPE), (dict(lddo=7), SHAPE), (dict(ldz=7), SHAPE), (dict(lddz=7), SHAPE), (dict(act=9), UNSUP),
        (dict(type=2), UNSUP), (dict(lddo=BIG), UNSUP), (dict(dO=None), NULL), (dict(Z=None), NULL),
        (dict(dZ=None, db=None), NULL), (dict(ws=None), NULL), (dict(ws=P(0x10008)), ALIGN),
        (dict(bytes=4 * 8 * 4 - 1), SHAPE), (dict(dO=P(0x10001)), ALIGN), (dict(Z=P(0x10001)), ALIGN),
        (dict(dZ=P(0x10001)), ALIGN), (dict(db=ODD), ALIGN), (dict(n=0, dO=None, lddo=0, ldz=0, lddz=0), OK),
        (dict(m=0, db=None, dO=None), OK)]],
])
def test_refusals(lib, fn, make, change, status):
    assert getattr(lib, fn)(*make(**change)) == status


def test_workspace_bytes(lib):
    n = ctypes.c_int64(7)
    for fn, per in (("kq_layernorm_backward_workspace_bytes", 8), ("kq_mxfp4_linear_backward_workspace_bytes", 4)):
        f = getattr(lib, fn)
        assert f(1, 100, ctypes.byref(n)) == kq.KQ_OK and n.value == 0  # one part: no workspace
        last = 0
        for m in (1, 2, 4, 5, 17, 100, 1000, 5000, 1 << 20, (1 << 31) - 1):  # whole parts, more rows never fewer
            assert f(m, 100, ctypes.byref(n)) == kq.KQ_OK and n.value >= last and n.value % (100 * per) == 0
            last = n.value
        assert 0 < last <= 512 * 100 * per
        assert f(0, 100, ctypes.byref(n)) == kq.KQ_OK and n.value == 0
        assert f(-1, 100, ctypes.byref(n)) == kq.KQ_ERR_SHAPE
        assert f(1, BIG, ctypes.byref(n)) == kq.KQ_ERR_UNSUPPORTED
        assert f(1, 1, None) == kq.KQ_ERR_NULL


def test_binding_refuses_host_tensors():
    x = torch.zeros(2, 64)
    with pytest.raises(TypeError):
        kq.layernorm(x)
    with pytest.raises(TypeError):
        kq.layernorm_backward(x, x, x[:, 0], x[:, 0])
    with pytest.raises(TypeError):
        kq.layernorm_quantize_mxfp4(x)
    with pytest.raises(TypeError):
        kq.mxfp4_linear(x, x, x, x)
    with pytest.raises(TypeError):
        kq.mxfp4_linear_backward(x)
