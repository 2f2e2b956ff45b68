"""What the gated product's 256 x 128 kernel works on and loads, on the CPU: a host-only build of csrc/kq_tileorder.hpp
with a checker (tests/native/gated_loads_check.cpp) that every column is covered once, that half tiles without a column are
no work, and that no load, those for a work that does not follow among them, leaves its operand or takes a scalar offset past
its count of bytes."""
import os
import shutil
import subprocess

import pytest

from tests import test_gpu_gated as gpu
from tests import test_gpu_gated_halves as halves

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def ask(tmp_path_factory):
    if shutil.which("g++") is None:
        pytest.skip("g++ not found")
    exe = str(tmp_path_factory.mktemp("loads") / "gated_loads_check")
    p = subprocess.run(["g++", "-std=c++17", "-O2", "-Wall", "-Werror", "-I",
                        os.path.join(ROOT, "mxfp4_activation_quantizer_amd", "csrc"),
                        os.path.join(ROOT, "tests", "native", "gated_loads_check.cpp"), "-o", exe],
                       capture_output=True, text=True)
    assert p.returncode == 0, p.stderr

    def f(products, cus=256):
        """[(kernel, works, empty halves, those on a workgroup with other works)] of the products (m, n, k, packed)."""
        text = "".join("%d %d %d %d %d %d\n" % (m, n, k, packed, k > 256 and (packed or k % 128 == 0), cus)
                       for m, n, k, packed in products)
        p = subprocess.run([exe], input=text, capture_output=True, text=True, timeout=120)
        assert p.returncode == 0, p.stdout[-500:]
        out = p.stdout.split("\n")[:-1]
        assert len(out) == len(products)
        return [tuple(int(x) for x in r.split()) for r in out]

    return f


@pytest.mark.parametrize("cus", [256, 80, 8])
def test_columns_and_loads(ask, cus):
    """Every width of a last column tile, one row tile to many, two stages to many, a partial one."""
    ask([(m, n, k, 0) for m in (1, 255, 256, 257, 2048, 8191) for n in (*range(1, 132), 2687, 2752, 2753, 5440, 5441, 11008)
         for k in (384, 512, 4096)], cus)


def test_gpu_tests_reach_empty_halves(ask):
    """The GPU tests' products of narrow last column tiles run on this kernel, with empty halves where they should be: alone
    on their workgroup and between other works."""
    rows = ask([(m, n, k, p) for m, n, k in halves.PRODUCTS for p in ((0, 1) if k % 256 == 0 else (0,))])
    assert all(kernel == 5 for kernel, *_ in rows)
    assert any(empty > passed for _, _, empty, passed in rows) and any(passed for _, _, _, passed in rows)
    assert any(empty == 0 for _, _, empty, _ in rows)
    ask([(m, n, k, 1) for m, n, k in gpu.BIG if k % 256 == 0])
