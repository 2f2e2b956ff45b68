"""GPU: the operators around the W4A4 product run together as a layer uses them -- norm into the
quantizer, product with its epilogue, and the way back -- on other streams, in captured graphs, and
against 64 bits with the quantizer held at the codes that the forward pass wrote."""
import numpy as np
import pytest

import synth
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


class Layer:
    """x -> x + gelu_tanh(deq(Q(LN(x) T)) deq(W)^T + bias), d = n, T block diagonal."""

    def __init__(self, torch, kq, d, seed):
        g = torch.Generator("cuda").manual_seed(seed)
        self.kq, self.d = kq, d
        self.weight = 1 + 0.1 * torch.randn(d, generator=g, device="cuda")
        self.beta = 0.1 * torch.randn(d, generator=g, device="cuda")
        self.bias = 0.1 * torch.randn(d, generator=g, device="cuda")
        f = synth.lu_perturbed_factors(d // 32, seed)
        self.factors = torch.from_numpy(f).cuda()
        w = torch.randn(d, d, generator=g, device="cuda") * d ** -0.5
        self.w = kq.quantize_mxfp4_f32(kq.inverse_fold_weights(w, self.factors))
        self.packed = d % 256 == 0
        self.sw = kq.pack_mxfp4_scales(self.w[1]) if self.packed else self.w[1]
        k = np.ones((d // 32, 1, 1))
        for i in range(5):
            k = np.stack([np.kron(a, b) for a, b in zip(k, f[:, i].astype(np.float64))])
        self.k = torch.from_numpy(k).cuda()

    def forward(self, x):
        kq = self.kq
        codes, scales, mean, rstd = kq.layernorm_quantize_mxfp4(x, self.weight, self.beta, self.factors, eps=EPS,
                                                                packed=self.packed, stats=True)
        out, z = kq.mxfp4_linear(codes, scales, self.w[0], self.sw, bias=self.bias, act="gelu_tanh", residual=x,
                                 bf16=x.dtype != self.weight.dtype, packed=self.packed, want_pre=True)
        return out, (codes, scales, mean, rstd, z)

    def token(self, x):
        """The serving form: no values kept for a backward pass."""
        kq = self.kq
        codes, scales = kq.layernorm_quantize_mxfp4(x, self.weight, self.beta, self.factors, eps=EPS,
                                                    packed=self.packed)
        return kq.mxfp4_linear(codes, scales, self.w[0], self.sw, bias=self.bias, act="gelu_tanh", residual=x,
                               bf16=x.dtype != self.weight.dtype, packed=self.packed)

    def backward(self, x, kept, dout, w32, kt):
        """Straight through the quantizer: d(y T) = dz deq(W), dy = d(y T) T^T, then the norm."""
        kq = self.kq
        _, _, mean, rstd, z = kept
        dz, dbias = kq.mxfp4_linear_backward(dout, z, act="gelu_tanh")
        dt = kq.gemm_f32(dz.float(), w32)
        dy = kq.gemm_f32(dt, kt)
        dx, dw, db = kq.layernorm_backward(dy.to(x.dtype), x, mean, rstd, self.weight)
        return dx + dout, dw, db, dbias


def block_diagonal(torch, k):
    d = 32 * k.shape[0]
    t = torch.zeros(d, d, dtype=torch.float64, device="cuda")
    for j in range(k.shape[0]):
        t[32 * j:32 * j + 32, 32 * j:32 * j + 32] = k[j]
    return t


@pytest.mark.parametrize("m,d", [(1, 512), (37, 544), (300, 1152), (600, 768)])
def test_forward_and_backward(torch, kq, m, d):
    layer = Layer(torch, kq, d, m)
    g = torch.Generator("cuda").manual_seed(m)
    x = torch.randn(m, d, generator=g, device="cuda") * 2 + 0.3
    dout = torch.randn(m, d, generator=g, device="cuda")
    out, kept = layer.forward(x)
    codes, scales, mean, rstd, z = kept
    sa = ref.unpack_scales(scales, m, d) if layer.packed else scales
    o, z64, o_tol, z_tol = ref.linear(codes, sa, layer.w[0], layer.w[1], layer.bias, "gelu_tanh", x)
    ref.assert_near(z, z64, z_tol, "z")
    ref.assert_near(out, o, o_tol, "out")
    assert torch.equal(layer.token(x), out)
    # the quantized activation stands for y T: no further from it than half a step of the largest
    # level (1 of 6) for every element of a block, whose maximum is at least 4 levels
    y = ref.norm(x, layer.weight, layer.beta, EPS)[0]
    t64 = block_diagonal(torch, layer.k)
    yt = (y @ t64).view(m, -1, 32)
    q = ref.decode(codes, sa).view(m, -1, 32)
    top = yt.abs().amax(2, keepdim=True)
    assert bool(((q - yt).abs() <= top * 0.25 + 1e-4).all())  # saturation: 6 stands for up to 8

    w64 = ref.decode(layer.w[0], layer.w[1])
    dx, dw, db, dbias = layer.backward(x, kept, dout, w64.float(), t64.t().float().contiguous())
    (dz, dbias64), (dz_tol, db_tol) = ref.linear_grad(dout, z, "gelu_tanh")
    ref.assert_near(dbias, dbias64, db_tol, "dbias")
    dy64 = dz @ w64 @ t64.t()
    want, tol = ref.norm_grad(dy64, x, mean, rstd, layer.weight)
    # the two fp32 products: (k + 2) 2^-22 of the sums of absolute values, through the norm's
    # backward, which is linear in dy with coefficients at most rstd |weight| (2 + |h| mean |h|)
    dt_tol = dz_tol @ w64.abs() + (d + 2) * 2.0 ** -22 * (dz.abs() @ w64.abs())
    dy_tol = dt_tol @ t64.abs().t() + (d + 2) * 2.0 ** -22 * ((dz @ w64).abs() @ t64.abs().t()) + 2 * ref.U * dy64.abs()
    h = (x.double() - mean.double()[:, None]) * rstd.double()[:, None]
    e = dy_tol * layer.weight.double().abs()
    dx_tol = tol[0] + rstd.double()[:, None] * (e + e.mean(1, keepdim=True) + h.abs() * (e * h.abs()).mean(1, keepdim=True))
    ref.assert_near(dx, want[0] + dout.double(), dx_tol + 2 * ref.U * (want[0].abs() + dout.abs()), "dx")
    ref.assert_near(dw, want[1], tol[1] + (dy_tol * h.abs()).sum(0), "dweight")
    ref.assert_near(db, want[2], tol[2] + dy_tol.sum(0), "dbias of the norm")


def all_ops(torch, kq, layer, x, dout):
    out, (codes, scales, mean, rstd, z) = layer.forward(x)
    y, mu, rs = kq.layernorm(x, layer.weight, layer.beta, stats=True)
    dz, dbias = kq.mxfp4_linear_backward(dout, z, act="gelu_tanh")
    dx, dw, db = kq.layernorm_backward(dz, x, mean, rstd, layer.weight)
    return [out, codes, scales, mean, rstd, z, y, mu, rs, dz, dbias, dx, dw, db]


@pytest.mark.parametrize("dt", ["bfloat16", "float32"])
def test_other_stream(torch, kq, dt):
    """Given a stream, a call runs and allocates on it: results as on the current stream, while both
    streams are kept busy and memory freed on one is taken again on the other."""
    layer = Layer(torch, kq, 768, 3)
    x = (torch.randn(500, 768, device="cuda") * 2).to(getattr(torch, dt))
    dout = torch.randn(500, 768, device="cuda").to(x.dtype)
    want = all_ops(torch, kq, layer, x, dout)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(5):
        y, mean, rstd = kq.layernorm(x, layer.weight, layer.beta, stats=True, stream=side)
        codes, scales, mu, rs = kq.layernorm_quantize_mxfp4(x, layer.weight, layer.beta, layer.factors, eps=EPS,
                                                            packed=True, stats=True, stream=side)
        out, z = kq.mxfp4_linear(codes, scales, layer.w[0], layer.sw, bias=layer.bias, act="gelu_tanh", residual=x,
                                 bf16=dt == "bfloat16", packed=True, want_pre=True, stream=side)
        dz, dbias = kq.mxfp4_linear_backward(dout, z, act="gelu_tanh", stream=side)
        dx, dw, db = kq.layernorm_backward(dz, x, mean, rstd, layer.weight, stream=side)
        got = [out, codes, scales, mu, rs, z, y, mean, rstd, dz, dbias, dx, dw, db]
        again = all_ops(torch, kq, layer, x, dout)  # beside it, on the current stream
        side.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        assert all(torch.equal(a, b) for a, b in zip(again, want))
        torch.cuda.synchronize()


def test_two_graphs_replayed(torch, kq):
    """Two captured graphs of the whole set, replayed in turn with eager calls between and then on two
    streams at once: each call's workspace is its own."""
    layer = Layer(torch, kq, 768, 4)
    xs = [(torch.randn(m, 768, device="cuda") * 2).bfloat16() for m in (200, 333)]
    ds = [torch.randn(m, 768, device="cuda").bfloat16() for m in (200, 333)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for x, d in zip(xs, ds):
            all_ops(torch, kq, layer, x, d)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graphs, outs = [], []
    for x, d in zip(xs, ds):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(all_ops(torch, kq, layer, x, d))
        graphs.append(g)
    for step in range(4):
        for x, d in zip(xs, ds):
            x.copy_((torch.randn(x.shape, device="cuda") * (1 + step)).bfloat16())
            d.copy_(torch.randn(d.shape, device="cuda").bfloat16())
        want = [all_ops(torch, kq, layer, x, d) for x, d in zip(xs, ds)]
        torch.cuda.synchronize()
        if step < 2:
            for g in graphs:
                g.replay()
                all_ops(torch, kq, layer, xs[0], ds[0])
        else:
            lanes = [torch.cuda.Stream(), torch.cuda.Stream()]
            for g, lane in zip(graphs, lanes):
                with torch.cuda.stream(lane):
                    g.replay()
        torch.cuda.synchronize()
        for got, w in zip(outs, want):
            assert all(torch.equal(a, b) for a, b in zip(got, w)), step


def test_backward_captured_while_an_eager_graph_lives(torch, kq):
    """The backward calls are plain launches: captured while torch's autograd holds an eager graph of the
    same leaves, they replay to the eager result."""
    x = torch.randn(64, 256, device="cuda", requires_grad=True)
    loss = (x * 2).sum()  # an eager graph of x that stays alive
    dy = torch.randn(64, 256, device="cuda")
    xd = x.detach()
    _, mean, rstd = kq.layernorm(xd, stats=True)
    want = kq.layernorm_backward(dy, xd, mean, rstd)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = kq.layernorm_backward(dy, xd, mean, rstd)
        dz = kq.mxfp4_linear_backward(dy, xd, act="silu")
    for _ in range(3):
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        assert all(torch.equal(a, b) for a, b in zip(dz, kq.mxfp4_linear_backward(dy, xd, act="silu")))
    loss.backward()
    assert bool((x.grad == 2).all())


@pytest.mark.parametrize("m,d", [(3, 515), (3, 1024), (300, 515), (300, 1024), (40, 16390)])
def test_each_gradient_alone(torch, kq, m, d):
    """The C entry points with one of the summed gradients, or with the sum alone: the values of the whole call,
    and nothing else written."""
    import ctypes
    L = kq.lib()
    x, dy = torch.randn(m, d, device="cuda"), torch.randn(m, d, device="cuda")
    w = torch.rand(d, device="cuda") + 0.5
    _, mean, rstd = kq.layernorm(x, w, stats=True)
    dx, dw, db = kq.layernorm_backward(dy, x, mean, rstd, w)
    n = ctypes.c_int64(0)
    assert L.kq_layernorm_backward_workspace_bytes(m, d, ctypes.byref(n)) == 0
    ws = torch.empty(max(n.value, 16), dtype=torch.uint8, device="cuda")
    stream = torch.cuda.current_stream().cuda_stream
    for which in (0, 1):
        got, gx = torch.full((d + 8,), 7.0, device="cuda"), torch.empty_like(x)
        out = got.data_ptr()
        assert L.kq_layernorm_backward(dy.data_ptr(), d, x.data_ptr(), d, 0, m, d, w.data_ptr(), mean.data_ptr(),
                                       rstd.data_ptr(), gx.data_ptr(), d, None if which else out, out if which else None,
                                       ws.data_ptr(), n.value, stream) == 0
        assert torch.equal(gx, dx) and torch.equal(got[:d], (dw, db)[which]) and bool((got[d:] == 7.0).all())
    dz, dbias = kq.mxfp4_linear_backward(dy, x, act="silu")
    assert L.kq_mxfp4_linear_backward_workspace_bytes(m, d, ctypes.byref(n)) == 0
    ws = torch.empty(max(n.value, 16), dtype=torch.uint8, device="cuda")
    got, gz = torch.full((d + 8,), 7.0, device="cuda"), torch.empty_like(x)
    silu = kq.ACTS["silu"]
    assert L.kq_mxfp4_linear_backward(dy.data_ptr(), d, x.data_ptr(), d, 0, m, d, silu, None, 0, got.data_ptr(),
                                      ws.data_ptr(), n.value, stream) == 0
    assert torch.equal(got[:d], dbias) and bool((got[d:] == 7.0).all())
    assert L.kq_mxfp4_linear_backward(dy.data_ptr(), d, x.data_ptr(), d, 0, m, d, silu, gz.data_ptr(), d, None, None, 0,
                                      stream) == 0
    assert torch.equal(gz, dz)


def test_two_streams_at_once(torch, kq):
    """Calls of every operator on two streams at the same time, each with its own workspace: each the values of a
    call alone."""
    m, d = 600, 1152
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    x = [torch.randn(m, d, device="cuda") for _ in streams]
    dy = torch.randn(m, d, device="cuda")
    w = torch.rand(d, device="cuda") + 0.5
    cw, sw = kq.quantize_mxfp4_f32(torch.randn(1000, d, device="cuda"))

    def run(v):
        y, mean, rstd = kq.layernorm(v, w, stats=True)
        codes, scales = kq.layernorm_quantize_mxfp4(v, w)
        o, z = kq.mxfp4_linear(codes, scales, cw, sw, act="gelu", want_pre=True, bf16=False)
        return (y, codes, scales, o, z) + kq.layernorm_backward(dy, v, mean, rstd, w) + \
            kq.mxfp4_linear_backward(o, z, act="gelu")

    want = [run(v) for v in x]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(5):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(run(x[i]))
    torch.cuda.synchronize()
    for i in range(2):
        for g in got[i]:
            assert all(torch.equal(a, b) for a, b in zip(g, want[i]))
