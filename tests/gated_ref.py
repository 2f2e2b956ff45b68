"""Plain 64-bit forms of kq_mxfp4_gated_linear and its gradients, and the error bounds of the fp32 kernels (test
infrastructure). The two products and the activations have the bounds of tests/layer_ref.py; for bf16 outputs
gelu's distribution function comes from a shorter polynomial, good to (45 + 1.2 z^2) 2^-24 of itself."""
import torch

from tests import layer_ref as ref

U = ref.U


def value(z, name, dtype):
    """(act(z), its slope, the kernels' own error in the value and in the slope at an exact z)"""
    a, slope = ref.act(z, name)
    v_tol, s_tol = ref.act_tol(z, name)
    if name == "gelu" and dtype == torch.bfloat16:
        v_tol = v_tol + (45 + 1.2 * z.clamp(-13, 13).square()) * U * a.abs()
    return a, slope, v_tol, s_tol


def forward(ca, sa, cg, sg, cu, su, bg, bu, name, dtype):
    """(out, g, u, and their bounds before the rounding)"""
    _, g, _, g_tol = ref.linear(ca, sa, cg, sg, bg, "none", None)
    _, u, _, u_tol = ref.linear(ca, sa, cu, su, bu, "none", None)
    a, _, v_tol, _ = value(g, name, dtype)
    a_tol = 1.2 * g_tol + v_tol  # no slope exceeds 1.13
    o = a * u
    return o, g, u, a_tol * (u.abs() + u_tol) + a.abs() * u_tol + 2 * U * o.abs(), g_tol, u_tol


def backward(dout, g, u, name):
    """((dg, du, dbias_g, dbias_u), their bounds before the rounding)"""
    dout, g, u = dout.double(), g.double(), u.double()
    a, slope, v_tol, s_tol = value(g, name, torch.float32)
    dg, du = dout * u * slope, dout * a
    dg_tol = (dout * u).abs() * s_tol + 3 * U * dg.abs()
    du_tol = dout.abs() * v_tol + 2 * U * du.abs()
    rows = dout.shape[0] / 16 + 512 + 24
    return ((dg, du, dg.sum(0), du.sum(0)),
            (dg_tol, du_tol, dg_tol.sum(0) + rows * U * dg.abs().sum(0), du_tol.sum(0) + rows * U * du.abs().sum(0)))
