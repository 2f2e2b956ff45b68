"""GPU: the gated product's 256 x 128 kernel where the last column tile is narrow, so that halves of it have no column
(tests/test_gated_loads.py holds these products to that kernel)."""
import pytest

from tests import test_gpu_gated as gated
from tests.test_gpu_gated import kq, torch  # noqa: F401  (fixtures)

pytestmark = pytest.mark.gpu

# halves alone on their workgroups and behind whole tiles; a last tile of 1, 52, 64 (a half's last one), 65 and 125 columns
PRODUCTS = [(1000, 2752, 2048), (1000, 2753, 2048), (2048, 5440, 2048), (2048, 5441, 1024), (2300, 5377, 1152), (4096, 2112, 1024),
            (4608, 2100, 1280), (8192, 1345, 1024)]


@pytest.mark.parametrize("m,n,k", PRODUCTS)
def test_narrow_last_tile(torch, kq, m, n, k):  # noqa: F811
    for i, packed in enumerate([False, True] if k % 256 == 0 else [False]):
        for j, dt in enumerate(("bfloat16", "float32")):
            gated.check(torch, kq, m, n, k, gated.ACTS[(m // 100 + n + 2 * i + j) % 5], dt, packed, bias=(i + j) % 2 == 0, seed=n,
                        pad=3 * (n % 2))
