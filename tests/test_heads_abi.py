"""The heads' entry points on the CPU: what they refuse before any HIP call, the frequencies, and the 64-bit forms
that the GPU tests use, against automatic differentiation and complex arithmetic."""
import ctypes
import math

import numpy as np
import pytest
import torch

import mxfp4_activation_quantizer_amd as kq
from tests import heads_ref as ref

P = ctypes.c_void_p
GOOD = P(0x10000)  # never dereferenced: every case below fails before a launch, or has nothing to do
BIG = 1 << 31


@pytest.fixture(scope="module")
def L():
    return kq.lib()


def rope(rot=64, axes=1, pairs=(32, 0, 0, 0), positions=0x10000, freq=0x10000):
    return ctypes.byref(kq._Rope(positions, freq, rot, 0, 1.0, axes, pairs))


def forward(X=GOOD, type=1, m=4, heads=6, d=64, ldx=384, hsx=64, norm=1, wq=GOOD, wk=GOOD, q=4, eps=1e-6, r=None, Y=GOOD,
            ldy=384, hsy=64):
    return ("kq_headnorm_rope", X, type, m, heads, d, ldx, hsx, norm, wq, wk, q, eps, r, Y, ldy, hsy, None)


def backward(dY=GOOD, X=GOOD, type=0, m=400, heads=6, d=64, norm=1, wq=GOOD, q=4, eps=1e-6, r=None, dX=GOOD, lddx=384, hsdx=64,
             dq=GOOD, dk=GOOD, ws=GOOD, ws_bytes=100 * 2 * 64 * 4, lddy=384, hsdy=64, ldx=384, hsx=64):
    return ("kq_headnorm_rope_backward", dY, lddy, hsdy, X, ldx, hsx, type, m, heads, d, norm, wq, wq, q, eps, r, dX, lddx, hsdx,
            dq, dk, ws, ws_bytes, None)


def write(K=GOOD, ldk=256, hsk=64, kh=2, V=GOOD, ldv=256, hsv=64, vh=2, type=1, m=4, d=64, norm=1, w=GOOD, eps=1e-6,
          r=None, slots=GOOD, n=9, ck=GOOD, sk=GOOD, cv=GOOD, sv=GOOD):
    return ("kq_cache_write_mxfp4", K, ldk, hsk, kh, V, ldv, hsv, vh, type, m, d, norm, w, eps, r, slots, n, ck, sk, cv, sv, None)


def read(slots=GOOD, m=4, codes=GOOD, scales=GOOD, n=9, heads=2, d=64, type=1, Y=GOOD, ldy=128, hsy=64):
    return ("kq_cache_read_mxfp4", slots, m, codes, scales, n, heads, d, type, Y, ldy, hsy, None)


SHAPE, NULL, ALIGN, UNSUPPORTED, OK = kq.KQ_ERR_SHAPE, kq.KQ_ERR_NULL, kq.KQ_ERR_ALIGN, kq.KQ_ERR_UNSUPPORTED, kq.KQ_OK


@pytest.mark.parametrize("call,status", [
    (forward(m=-1), SHAPE), (forward(heads=-1), SHAPE), (forward(d=-64), SHAPE), (forward(q=7), SHAPE), (forward(q=-1), SHAPE),
    (forward(ldx=-1), SHAPE), (forward(hsx=-1), SHAPE), (forward(eps=-1.0), SHAPE), (forward(eps=math.nan), SHAPE),
    (forward(eps=math.inf), SHAPE), (forward(type=2), UNSUPPORTED), (forward(d=1025, ldy=7000, hsy=1025), UNSUPPORTED),
    (forward(heads=65537), UNSUPPORTED), (forward(m=BIG), UNSUPPORTED), (forward(ldx=BIG), UNSUPPORTED),
    (forward(hsy=63), SHAPE), (forward(ldy=383), SHAPE), (forward(ldy=64, hsy=255), SHAPE), (forward(ldy=0, hsy=0), SHAPE),
    (forward(X=None), NULL), (forward(Y=None), NULL), (forward(X=P(0x10001)), ALIGN), (forward(Y=P(0x10001)), ALIGN),
    (forward(wq=P(0x10002)), ALIGN), (forward(wk=P(0x10001)), ALIGN), (forward(m=0, X=None, Y=None), OK),
    (forward(heads=0, q=0, X=None, Y=None), OK), (forward(d=0, X=None, Y=None), OK),
    (forward(r=rope(rot=63)), SHAPE), (forward(r=rope(rot=66)), SHAPE), (forward(r=rope(rot=-2)), SHAPE),
    (forward(r=rope(axes=0)), UNSUPPORTED), (forward(r=rope(axes=5)), UNSUPPORTED), (forward(r=rope(pairs=(31, 1, 0, 0))), SHAPE),
    (forward(r=rope(axes=2, pairs=(40, -8, 0, 0))), SHAPE), (forward(r=rope(axes=2, pairs=(1 << 62, 1 << 62, 0, 0))), SHAPE),
    (forward(r=rope(positions=None)), NULL), (forward(r=rope(freq=None)), NULL), (forward(r=rope(positions=0x10004)), ALIGN),
    (forward(r=rope(freq=0x10004)), ALIGN), (forward(m=0, r=rope(positions=None, freq=None)), OK),
    (backward(m=-1), SHAPE), (backward(lddy=-1), SHAPE), (backward(norm=0), SHAPE), (backward(eps=-1e-9), SHAPE),
    (backward(type=-1), UNSUPPORTED), (backward(d=2048, lddx=12288, hsdx=2048), UNSUPPORTED), (backward(hsdx=60), SHAPE),
    (backward(dY=None), NULL), (backward(X=None), NULL), (backward(dX=None), NULL), (backward(ws=None), NULL),
    (backward(ws=P(0x10008)), ALIGN), (backward(ws_bytes=51199), SHAPE), (backward(dY=P(0x10002)), ALIGN),
    (backward(X=P(0x10002)), ALIGN), (backward(dX=P(0x10002)), ALIGN), (backward(dq=P(0x10002)), ALIGN),
    (backward(wq=P(0x10002)), ALIGN), (backward(r=rope(rot=30)), SHAPE), (backward(q=8), SHAPE),
    (backward(m=0, dq=None, dk=None, dY=None, X=None, dX=None), OK), (backward(d=0), OK),
    (write(d=48), SHAPE), (write(m=-1), SHAPE), (write(n=-1), SHAPE), (write(kh=-1), SHAPE), (write(vh=-1), SHAPE), (write(ldk=-1), SHAPE),
    (write(hsv=-1), SHAPE), (write(eps=-1.0), SHAPE), (write(type=3), UNSUPPORTED), (write(d=1056), UNSUPPORTED),
    (write(kh=65535), UNSUPPORTED), (write(n=BIG), UNSUPPORTED), (write(slots=None), NULL), (write(K=None), NULL), (write(V=None), NULL),
    (write(ck=None), NULL), (write(sv=None), NULL), (write(slots=P(0x10004)), ALIGN), (write(ck=P(0x10002)), ALIGN),
    (write(cv=P(0x10001)), ALIGN), (write(K=P(0x10001)), ALIGN), (write(V=P(0x10001)), ALIGN), (write(w=P(0x10002)), ALIGN),
    (write(r=rope(rot=62)), SHAPE), (write(m=0, K=None), OK), (write(n=0), OK), (write(kh=0, vh=0), OK), (write(d=0), OK),
    (write(m=0, kh=0, K=None, ck=None, sk=None, ldk=-5, r=rope(rot=62)), OK),
    (read(d=40), SHAPE), (read(m=-1), SHAPE), (read(n=-1), SHAPE), (read(heads=-1), SHAPE), (read(ldy=127), SHAPE), (read(ldy=-1), SHAPE),
    (read(type=9), UNSUPPORTED), (read(d=2048, hsy=2048, ldy=4096), UNSUPPORTED), (read(heads=BIG), UNSUPPORTED),
    (read(slots=None), NULL), (read(Y=None), NULL), (read(codes=None), NULL), (read(scales=None), NULL), (read(codes=P(0x10002)), ALIGN),
    (read(slots=P(0x10001)), ALIGN), (read(Y=P(0x10001)), ALIGN), (read(m=0, Y=None, slots=None), OK), (read(heads=0), OK),
    (read(d=0), OK),
])
def test_host_argument_checks(L, call, status):
    assert getattr(L, call[0])(*call[1:]) == status


def test_workspace_bytes(L):
    n = ctypes.c_int64(-1)
    for m, d, want in ((0, 64, 0), (4, 64, 0), (5, 64, 2 * 2 * 64 * 4), (1 << 20, 1024, 256 * 2 * 1024 * 4), (9, 0, 0)):
        assert L.kq_headnorm_rope_backward_workspace_bytes(m, d, ctypes.byref(n)) == OK and n.value == want
    assert L.kq_headnorm_rope_backward_workspace_bytes(4, 64, None) == NULL
    assert L.kq_headnorm_rope_backward_workspace_bytes(-1, 64, ctypes.byref(n)) == SHAPE
    assert L.kq_headnorm_rope_backward_workspace_bytes(4, 1025, ctypes.byref(n)) == UNSUPPORTED
    assert L.kq_headnorm_rope_backward_workspace_bytes(BIG, 4, ctypes.byref(n)) == UNSUPPORTED


def test_frequencies():
    i = np.arange(32)
    plain = kq.rope_frequencies(64, 10000.0)
    assert np.allclose(plain, 10000.0 ** (-i / 32), rtol=1e-14, atol=0)
    assert np.allclose(kq.rope_frequencies(64, scaling="linear", factor=8.0), plain / 8, rtol=1e-14, atol=0)
    base = kq.rope_frequencies(64, scaling="base", factor=8.0)
    assert base[0] == 1 and math.isclose(base[-1], plain[-1] / 8, rel_tol=1e-12)
    assert np.allclose(base, (10000.0 * 8 ** (64 / 62)) ** (-i / 32), rtol=1e-13, atol=0)
    parts = kq.rope_frequencies(64, scaling="parts", factor=8.0, original=4096, low=1, high=32)
    turns = 4096 * plain / (2 * np.pi)
    assert np.array_equal(parts[turns > 32], plain[turns > 32])
    assert np.allclose(parts[turns < 1], plain[turns < 1] / 8, rtol=1e-14, atol=0)
    between = (turns >= 1) & (turns <= 32)
    assert between.any()
    keep = (turns[between] - 1) / 31
    assert np.allclose(parts[between], plain[between] * (keep + (1 - keep) / 8), rtol=1e-13, atol=0)
    assert kq.rope_frequencies(2, scaling="base", factor=8.0)[0] == 1 and kq.rope_frequencies(0).size == 0
    for bad in (dict(rot=3), dict(rot=-2), dict(rot=4, base=0.0), dict(rot=4, base=math.nan), dict(rot=4, scaling="linear", factor=0.0),
                dict(rot=4, scaling="parts", factor=2.0), dict(rot=4, scaling="parts", factor=2.0, original=9.0, low=2, high=2)):
        with pytest.raises(kq.KQError):
            kq.rope_frequencies(**bad)
    with pytest.raises(ValueError):
        kq.rope_frequencies(4, scaling="other")


@pytest.mark.parametrize("inter", [False, True])
def test_the_64_bit_forms(inter):
    """The gradients by automatic differentiation of the forward form, and that by complex numbers."""
    g = torch.Generator().manual_seed(3)
    m, heads, q, d = 7, 5, 3, 12
    x, dy = (torch.randn(m, heads, d, generator=g, dtype=torch.float64) for _ in range(2))
    wq, wk = (torch.randn(d, generator=g, dtype=torch.float64) for _ in range(2))
    r = {"positions": torch.randint(-50, 50, (m, 2), generator=g), "freq": torch.rand(4, generator=g, dtype=torch.float64),
         "inter": inter, "axis_pairs": (3, 1), "amplitude": 1.3}
    leaves = [t.clone().requires_grad_() for t in (x, wq, wk)]
    y, tol = ref.forward(*leaves, q, 1e-6, r)
    y.backward(dy)
    got, tols = ref.backward(dy, x, wq, wk, q, 1e-6, r)
    for a, b, t in zip(got, leaves, tols):
        assert torch.allclose(a, b.grad, rtol=1e-11, atol=1e-12)
        assert bool((t > 0).all())
    assert bool((tol > 0).all()) and bool((tol < 1e-4).all())
    n = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6) * torch.cat((wq.expand(q, -1), wk.expand(heads - q, -1)))
    for i in range(4):
        a, b = (2 * i, 2 * i + 1) if inter else (i, i + 4)
        t = r["positions"][:, 0 if i < 3 else 1].double() * r["freq"][i]
        z = torch.complex(n[..., a], n[..., b]) * torch.polar(torch.full_like(t, 1.3), t)[:, None]
        assert torch.allclose(y[..., a], z.real) and torch.allclose(y[..., b], z.imag)
    assert torch.allclose(y[..., 8:], n[..., 8:])


def test_the_code_check_rejects_mistakes(orc):
    g = torch.Generator().manual_seed(5)
    y = torch.randn(9, 64, generator=g, dtype=torch.float64)
    tol = 1e-6 * y.abs()
    codes, scales = (torch.from_numpy(np.asarray(t)) for t in orc.quantize_f32(y.float().numpy()))
    ref.assert_codes_near(codes, scales, y, tol)
    for mistake in ("code", "scale", "sign"):
        c, s = codes.clone(), scales.clone()
        if mistake == "scale":
            s[4, 1] += 1
        else:
            c[4, 7] ^= 1 if mistake == "code" else 8
        with pytest.raises(AssertionError):
            ref.assert_codes_near(c, s, y, tol)


def test_packed_rotation():
    """The binding's bytes of a kq_rope are the structure's."""
    r = kq._Rope(1 << 40, 1 << 41, 64, 1, 1.5, 3, (20, 10, 2, 0))
    assert kq._ROPE.pack(1 << 40, 1 << 41, 64, 1, 1.5, 3, 20, 10, 2, 0) == bytes(r)
