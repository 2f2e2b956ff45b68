"""GPU: the rotation's angles as the header states them, p freq[i] off by 2^-51 of itself for any position, against exact
arithmetic."""
import math
import random
from fractions import Fraction

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


def two_pi(bits=400):
    """2 pi to `bits` bits, by pi / 4 = 4 atan(1/5) - atan(1/239)."""
    one = 1 << (bits + 16)

    def atan_of_1_over(n):
        total, term, i = 0, one // n, 1
        while term:
            total += term // i if i % 4 == 1 else -(term // i)
            term //= n * n
            i += 2
        return total

    return Fraction(8 * (4 * atan_of_1_over(5) - atan_of_1_over(239)), one)


def exact_turn(p, f, period):
    """(cos, sin) of p f, p an integer and f a double, the product reduced exactly."""
    t = Fraction(f) * p
    t -= round(t / period) * period
    return math.cos(float(t)), math.sin(float(t))


@pytest.mark.parametrize("size", [10, 24, 34, 44, 50, 56, 62])
@pytest.mark.parametrize("inter", [False, True])
def test_angles_of_far_positions(torch, kq, size, inter):
    r, period = random.Random(size), two_pi()
    m, n = 48, 24
    positions = [r.choice((-1, 1)) * r.randrange(1 << (size - 1), 1 << size) for _ in range(m - 3)]
    positions += [0, (1 << size) - 1, -(1 << size)]
    freq = [1.0] + [math.exp(-r.uniform(0, 14)) for _ in range(n - 1)]
    x = torch.zeros(m, 1, 2 * n, device="cuda")
    x[..., 0:2 * n:2 if inter else 1][..., :n] = 1.0  # each pair (1, 0): its turn is (cos, sin)
    y = kq.headnorm_rope(x, torch.tensor(positions, device="cuda"), torch.tensor(freq, dtype=torch.float64, device="cuda"),
                         norm=False, interleaved=inter)[:, 0].double().cpu()
    cos, sin = (y[:, 0::2], y[:, 1::2]) if inter else (y[:, :n], y[:, n:])
    for i, p in enumerate(positions):
        for j, f in enumerate(freq):
            c, s = exact_turn(p, f, period)
            # the angle's bound, then 1.5 units in the last place of a value of at most 1
            off = 2.0 ** -51 * abs(p) * f + 1.5 * 2.0 ** -23
            assert abs(float(cos[i, j]) - c) <= off and abs(float(sin[i, j]) - s) <= off, (p, f)
