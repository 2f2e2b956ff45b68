"""kq_mxfp4_gated_linear's entry points on the CPU: what they refuse before any HIP call, and the 64-bit forms that the
GPU tests use, against automatic differentiation."""
import ctypes

import pytest
import torch

import mxfp4_activation_quantizer_amd as kq
from tests import gated_ref as ref

P = ctypes.c_void_p
GOOD = P(0x10000)  # never dereferenced: every case below fails before a launch, or has nothing to do
BIG = 1 << 31
SHAPE, NULL, ALIGN, UNSUPPORTED, OK = kq.KQ_ERR_SHAPE, kq.KQ_ERR_NULL, kq.KQ_ERR_ALIGN, kq.KQ_ERR_UNSUPPORTED, kq.KQ_OK


def forward(ca=GOOD, sa=GOOD, cg=GOOD, sg=GOOD, cu=GOOD, su=GOOD, packed=0, m=4, n=8, k=256, bg=GOOD, bu=GOOD, act=2, type=1,
            O=GOOD, ldo=8, G=GOOD, ldg=8, U=GOOD, ldu=8):
    return ("kq_mxfp4_gated_linear", ca, sa, cg, sg, cu, su, packed, m, n, k, bg, bu, act, type, O, ldo, G, ldg, U, ldu, None)


def backward(dO=GOOD, lddo=8, G=GOOD, ldg=8, U=GOOD, ldu=8, type=0, m=40, n=8, act=2, dG=GOOD, lddg=8, dU=GOOD, lddu=8, bg=GOOD,
             bu=GOOD, ws=GOOD, ws_bytes=10 * 2 * 8 * 4):
    return ("kq_mxfp4_gated_linear_backward", dO, lddo, G, ldg, U, ldu, type, m, n, act, dG, lddg, dU, lddu, bg, bu, ws, ws_bytes, None)


@pytest.mark.parametrize("call,status", [
    (forward(m=-1), SHAPE), (forward(n=-1), SHAPE), (forward(k=-32), SHAPE), (forward(k=48), SHAPE), (forward(packed=1, k=128), SHAPE),
    (forward(ldo=7), SHAPE), (forward(ldg=7), SHAPE), (forward(ldu=7), SHAPE), (forward(G=None, ldg=0, m=0), OK),
    (forward(act=5), UNSUPPORTED), (forward(act=-1), UNSUPPORTED), (forward(type=2), UNSUPPORTED), (forward(m=BIG), UNSUPPORTED),
    (forward(n=BIG, ldo=BIG, ldg=BIG, ldu=BIG), UNSUPPORTED), (forward(k=BIG), UNSUPPORTED), (forward(ldo=BIG), UNSUPPORTED),
    (forward(ldg=BIG), UNSUPPORTED), (forward(ldu=BIG), UNSUPPORTED), (forward(k=1 << 24), UNSUPPORTED),
    (forward(m=1 << 28), UNSUPPORTED), (forward(n=1 << 28, ldo=1 << 28, ldg=1 << 28, ldu=1 << 28), UNSUPPORTED),
    (forward(ldo=1 << 23), UNSUPPORTED), (forward(ldg=1 << 23), UNSUPPORTED), (forward(ldu=1 << 23), UNSUPPORTED),
    (forward(ca=None), NULL), (forward(sa=None), NULL), (forward(cg=None), NULL), (forward(sg=None), NULL), (forward(cu=None), NULL),
    (forward(su=None), NULL), (forward(O=None), NULL), (forward(ca=P(0x10008)), ALIGN), (forward(cg=P(0x10008)), ALIGN),
    (forward(cu=P(0x10008)), ALIGN), (forward(packed=1, sa=P(0x10004)), ALIGN), (forward(packed=1, sg=P(0x10004)), ALIGN),
    (forward(packed=1, su=P(0x10004)), ALIGN), (forward(bg=P(0x10002)), ALIGN), (forward(bu=P(0x10002)), ALIGN),
    (forward(O=P(0x10001)), ALIGN), (forward(G=P(0x10001)), ALIGN), (forward(U=P(0x10001)), ALIGN),
    (forward(m=0, ca=None, O=None), OK), (forward(n=0, cg=None, O=None), OK),
    (backward(m=-1), SHAPE), (backward(n=-1), SHAPE), (backward(lddo=7), SHAPE), (backward(ldg=7), SHAPE), (backward(ldu=7), SHAPE),
    (backward(lddg=7), SHAPE), (backward(lddu=7), SHAPE), (backward(m=400, ws_bytes=6399), SHAPE), (backward(act=9), UNSUPPORTED),
    (backward(type=-1), UNSUPPORTED), (backward(m=BIG), UNSUPPORTED), (backward(lddu=BIG), UNSUPPORTED), (backward(dO=None), NULL),
    (backward(G=None), NULL), (backward(U=None), NULL), (backward(m=400, ws=None, ws_bytes=6400), NULL), (backward(dG=None, dU=None, bg=None, bu=None), NULL),
    (backward(dO=P(0x10002)), ALIGN), (backward(G=P(0x10002)), ALIGN), (backward(U=P(0x10002)), ALIGN), (backward(dG=P(0x10002)), ALIGN),
    (backward(dU=P(0x10002)), ALIGN), (backward(bg=P(0x10002)), ALIGN), (backward(bu=P(0x10001)), ALIGN), (backward(m=400, ws=P(0x10008), ws_bytes=6400), ALIGN),
    (backward(n=0, dO=None), OK), (backward(m=0, dO=None, bg=None, bu=None), OK),
])
def test_host_argument_checks(call, status):
    assert getattr(kq.lib(), call[0])(*call[1:]) == status


def test_workspace_bytes():
    n = ctypes.c_int64(-1)
    ask = kq.lib().kq_mxfp4_gated_linear_backward_workspace_bytes
    one = ctypes.c_int64(-1)
    for m, cols in ((0, 8), (4, 8), (301, 4607), (384, 8), (385, 8), (8192, 11008), (400, 0), (9, 0), (0, 0), (BIG - 1, BIG - 1),
                    (384, 1 << 26), (3, 1 << 28), (384, 1 << 28)):
        assert ask(m, cols, ctypes.byref(n)) == OK
        kq.lib().kq_mxfp4_linear_backward_workspace_bytes(m, cols, ctypes.byref(one))
        # up to 384 rows one workgroup sums all rows of a column
        assert n.value == (2 * one.value if m > 384 or cols >= 1 << 27 else 0)
    assert ask(4, 4, None) == NULL and ask(-1, 4, ctypes.byref(n)) == SHAPE and ask(4, BIG, ctypes.byref(n)) == UNSUPPORTED


@pytest.mark.parametrize("name", ["none", "relu", "silu", "gelu", "gelu_tanh"])
def test_the_64_bit_forms(name):
    g = torch.Generator().manual_seed(1)
    leaves = [torch.randn(7, 5, generator=g, dtype=torch.float64).requires_grad_() for _ in range(2)]
    dout = torch.randn(7, 5, generator=g, dtype=torch.float64)
    f = torch.nn.functional
    act = {"none": lambda z: z, "relu": f.relu, "silu": f.silu, "gelu": f.gelu, "gelu_tanh": lambda z: f.gelu(z, approximate="tanh")}[name]
    (act(leaves[0]) * leaves[1]).backward(dout)
    got, tol = ref.backward(dout, leaves[0].detach(), leaves[1].detach(), name)
    for i in range(2):
        assert torch.allclose(got[i], leaves[i].grad, rtol=1e-11, atol=1e-12)
        assert torch.allclose(got[2 + i], leaves[i].grad.sum(0), rtol=1e-11, atol=1e-12)
    assert all(bool((t < 1e-3).all()) for t in tol)
