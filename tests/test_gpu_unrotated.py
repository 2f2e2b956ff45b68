"""GPU: channels that no pair is in keep their bits, to the sign of a zero, so that keys that are neither normed nor
turned go into the cache with the oracle's bytes, at ties between two codes too."""
import math

import pytest

pytestmark = pytest.mark.gpu


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


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("d,rot", [(128, 64), (128, 0), (96, 32), (72, 24), (80, 16), (45, 12), (33, 0), (1024, 512), (20, 8)])
def test_channels_without_a_pair(torch, kq, d, rot, inter, dtype):
    """Zeros of both signs, infinities and ordinary values of the channels behind the rotated ones, forwards and back."""
    g = torch.Generator().manual_seed(d + rot)
    m, heads = 70, 5
    x = torch.randn(m, heads, d, generator=g).to(getattr(torch, dtype))
    odd = torch.tensor([0.0, -0.0, math.inf, -math.inf, 1.0, -1.0]).to(x.dtype)
    x[..., rot:] = torch.where(torch.rand(m, heads, d - rot, generator=g) < 0.7,
                               odd[torch.randint(0, 6, (m, heads, d - rot), generator=g)], x[..., rot:])
    x = x.cuda()
    rope = dict(positions=torch.arange(m, device="cuda"), interleaved=inter,
                freq=torch.logspace(0, -4, rot // 2, dtype=torch.float64, device="cuda"), amplitude=1.5) if rot else {}
    bits = torch.int16 if dtype == "bfloat16" else torch.int32
    y = kq.headnorm_rope(x, norm=False, **rope)
    dx, _, _ = kq.headnorm_rope_backward(x, norm=False, **rope)
    for got in (y, dx):
        assert torch.equal(got[..., rot:].contiguous().view(bits), x[..., rot:].contiguous().view(bits))
        assert bool(got[..., :rot].isfinite().all())


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
@pytest.mark.parametrize("heads,d", [(8, 128), (2, 64), (3, 96), (1, 32), (2, 160)])
def test_cache_at_ties(torch, kq, orc, heads, d, dtype):
    """Keys and values of nothing but zeros, borders between two codes and levels, in blocks of all scales: the oracle's
    bytes, in the form that quantizes in registers and in the staged one."""
    g = torch.Generator().manual_seed(d)
    m = 64
    of = torch.tensor([0.0, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, 7.0])
    v = of[torch.randint(0, 16, (m, heads, d), generator=g)]
    v = torch.where(torch.rand(v.shape, generator=g) < 0.5, -v, v)
    scale = torch.randint(-30, 31, (m, heads, d // 32, 1), generator=g)
    v = (v.view(m, heads, d // 32, 32).double() * 2.0 ** scale.double()).view(m, heads, d).to(getattr(torch, dtype))
    flat = v.float().view(m * heads, d).numpy()
    codes, scales = orc.quantize_f32(flat)
    slots = torch.randperm(m, generator=g)
    t = v.cuda()
    c = torch.zeros(2, m, heads, d // 2, dtype=torch.uint8, device="cuda")
    s = torch.zeros(2, m, heads, d // 32, dtype=torch.uint8, device="cuda")
    kq.cache_write_mxfp4(slots.cuda(), k=t, codes_k=c[0], scales_k=s[0], v=t, codes_v=c[1], scales_v=s[1])
    for i in range(2):
        assert torch.equal(c[i].cpu()[slots].view(m * heads, -1), torch.from_numpy(codes)), "kv"[i]
        assert torch.equal(s[i].cpu()[slots].view(m * heads, -1), torch.from_numpy(scales)), "kv"[i]
