"""GPU: calls of the heads' and the cache's entry points that mix what others keep alike: unlike numbers of key and value
heads, unlike strides and alignment of the two, vectors at addresses of 4 bytes, gradients in the place of either input."""
import math

import pytest

from tests import heads_ref as ref
from tests import layer_ref
from tests.test_gpu_heads import EPS, call_args, kq, make_heads, make_rope, torch  # noqa: F401  (fixtures)

pytestmark = pytest.mark.gpu


def vector(torch, g, d, shift):  # noqa: F811
    """1 and a little, `shift` floats behind an aligned address."""
    v = torch.empty(d + shift, device="cuda")[shift:]
    return v.copy_(1 + 0.2 * torch.randn(d, generator=g, device="cuda"))


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
@pytest.mark.parametrize("m,kh,vh,d,rot,inter", [(33, 2, 5, 128, 128, False), (7, 17, 1, 64, 64, True), (300, 1, 9, 32, 32, False),
                                                 (5, 33, 3, 96, 48, False), (1, 3, 64, 160, 160, True), (70, 1, 2, 1024, 512, False),
                                                 (2000, 3, 1, 32, 0, False)])
def test_unlike_keys_and_values(torch, kq, m, kh, vh, d, rot, inter, dtype):  # noqa: F811
    """Together as each alone: other numbers of heads, values transposed and a few elements off the keys' alignment."""
    dtype = getattr(torch, dtype)
    g = torch.Generator("cuda").manual_seed(m + d)
    k = make_heads(torch, g, m, kh, d, dtype)
    vs = torch.empty(vh * m * (d + 3) + 1, dtype=dtype, device="cuda")[1:].view(vh, m, d + 3)[:, :, :d].transpose(0, 1)
    vs.copy_(make_heads(torch, g, m, vh, d, dtype))
    w, rope, n = vector(torch, g, d, 1), make_rope(torch, g, m, rot, inter), m + 9
    slots = torch.randperm(n, generator=torch.Generator().manual_seed(m))[:m].cuda()

    def caches():
        return [torch.full((n, h, c), 0x55, dtype=torch.uint8, device="cuda") for h in (kh, vh) for c in (d // 2, d // 32)]

    both, alone = caches(), caches()
    key = dict(norm=True, weight=w, eps=EPS, **call_args(rope))
    kq.cache_write_mxfp4(slots, k=k, codes_k=both[0], scales_k=both[1], v=vs, codes_v=both[2], scales_v=both[3], **key)
    kq.cache_write_mxfp4(slots, v=vs.contiguous(), codes_v=alone[2], scales_v=alone[3])
    for a, b in zip(both[2:], alone[2:]):
        assert torch.equal(a, b)
    y, tol = ref.forward(k, w, w, kh, EPS, rope)
    ref.assert_codes_near(both[0][slots], both[1][slots], y, tol, "keys")
    rest = torch.ones(n, dtype=torch.bool, device="cuda")
    rest[slots] = False
    assert all(bool((t[rest] == 0x55).all()) for t in both)


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
@pytest.mark.parametrize("m,heads,q,d,rot,inter", [(200, 6, 4, 128, 128, False), (9, 5, 2, 72, 72, True), (40, 3, 1, 65, 64, False),
                                                   (1, 40, 32, 128, 64, False), (1030, 4, 3, 96, 96, False)])
def test_gradients_in_either_place(torch, kq, m, heads, q, d, rot, inter, dtype):  # noqa: F811
    """dx in the place of dy or of x, inside a fused product's rows; weights and their gradients at addresses of 4 bytes."""
    dtype = getattr(torch, dtype)
    g = torch.Generator("cuda").manual_seed(m + d)
    x, dy = (make_heads(torch, g, m, heads, d, dtype) for _ in range(2))
    wq, wk = vector(torch, g, d, 1), vector(torch, g, d, 3)
    rope = make_rope(torch, g, m, rot, inter)
    kw = dict(weight_q=wq, weight_k=wk, q_heads=q, eps=EPS, **call_args(rope))
    want, tol = ref.backward(dy, x, wq, wk, q, EPS, rope)
    for place in ("x", "dy"):
        rooms = {}
        for name, t in (("x", x), ("dy", dy)):
            rooms[name] = torch.full((m, heads + 2, d), math.nan, dtype=dtype, device="cuda")
            rooms[name][:, 1:heads + 1] = t
        views = {name: r[:, 1:heads + 1] for name, r in rooms.items()}
        dq, dk = (torch.empty(d + 1, device="cuda")[1:] for _ in range(2))
        dx, _, _ = kq.headnorm_rope_backward(views["dy"], views["x"], dx=views[place], dweight_q=dq, dweight_k=dk, **kw)
        assert dx is views[place]
        for a, b, t in zip((dx, dq, dk), want, tol):
            layer_ref.assert_near(a, b, t, place)
        other = "dy" if place == "x" else "x"
        assert torch.equal(views[other], dy if other == "dy" else x)
        for r in rooms.values():
            assert bool(r[:, 0].isnan().all()) and bool(r[:, -1].isnan().all())


@pytest.mark.parametrize("m,n", [(5, 40), (300, 1000), (385, 1000), (2000, 513)])
def test_gated_gradients_in_every_place(torch, kq, m, n):  # noqa: F811
    """dg and du in the places of any two of the three inputs, vectors at addresses of 4 bytes."""
    g0 = torch.Generator("cuda").manual_seed(m)
    ins = [torch.randn(m, n, generator=g0, device="cuda").to(torch.bfloat16) for _ in range(3)]
    want = kq.mxfp4_gated_linear_backward(*ins, act="gelu_tanh")
    for a in range(3):
        for b in range(3):
            if a == b:
                continue
            t = [x.clone() for x in ins]
            bg, bu = (torch.empty(n + 1, device="cuda")[1:] for _ in range(2))
            got = kq.mxfp4_gated_linear_backward(*t, act="gelu_tanh", dg=t[a], du=t[b], dbias_g=bg, dbias_u=bu)
            assert all(torch.equal(x, y) for x, y in zip(got, want)), (a, b)


def test_missing_parts_of_a_cache(torch, kq):  # noqa: F811
    """A tensor without its codes or scales, slots that are no tensor: refused by name, and nothing is written."""
    x = torch.ones(4, 2, 64, device="cuda")
    codes, scales = torch.zeros(9, 2, 32, dtype=torch.uint8, device="cuda"), torch.zeros(9, 2, 2, dtype=torch.uint8, device="cuda")
    slots = torch.arange(4, device="cuda")
    for kw in (dict(v=x, scales_v=scales), dict(v=x, codes_v=codes), dict(k=x, codes_k=codes), dict(k=x),
               dict(k=x, codes_k=codes, scales_k=scales, v=x)):
        with pytest.raises(ValueError, match="are required"):
            kq.cache_write_mxfp4(slots, **kw)
    for bad in (None, [0, 1, 2, 3]):
        with pytest.raises(TypeError, match="slots"):
            kq.cache_write_mxfp4(bad, v=x, codes_v=codes, scales_v=scales)
        with pytest.raises(TypeError, match="slots"):
            kq.cache_read_mxfp4(bad, codes, scales)
    with pytest.raises(ValueError, match="are required"):
        kq.cache_read_mxfp4(slots, codes, None)
    torch.cuda.synchronize()
    assert not codes.any() and not scales.any()
