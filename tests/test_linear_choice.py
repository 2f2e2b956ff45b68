"""Which kernel of kq_mxfp4_linear the GPU tests' products run on, on the CPU: a host-only build of the choice
(csrc/kq_choice.hpp, tests/native/choice_check.cpp) at 256 compute units. A refit of its estimates that would
leave a kernel, or a way through one, without a test fails here."""
import os
import shutil
import subprocess

import pytest

from tests import test_gpu_linear as gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
KERNELS = ["16 x 16", "16 x 32", "32 x 32", "64 x 64 deep", "64 x 64", "128 x 128", "256 x 256"]
TILE = {"16 x 16": (16, 16), "16 x 32": (16, 32), "32 x 32": (32, 32), "64 x 64 deep": (64, 64), "64 x 64": (64, 64),
        "128 x 128": (128, 128), "256 x 256": (256, 256)}


@pytest.fixture(scope="module")
def ask(tmp_path_factory):
    if shutil.which("g++") is None:
        pytest.skip("g++ not found")
    exe = str(tmp_path_factory.mktemp("choice") / "choice_check")
    p = subprocess.run(["g++", "-std=c++17", "-O2", "-Wall", "-Werror", "-I",
                        os.path.join(ROOT, "mxfp4_activation_quantizer_amd", "csrc"),
                        os.path.join(ROOT, "tests", "native", "choice_check.cpp"), "-o", exe],
                       capture_output=True, text=True)
    assert p.returncode == 0, p.stderr

    def f(products):
        """[(kernel, whole tiles, halved tiles)] of the products (m, n, k, packed)."""
        text = "".join("%d %d %d %d %d 256\n" % (m, n, (k + 255) // 256, packed, k > 0 and (packed or k % 128 == 0))
                       for m, n, k, packed in products)
        out = subprocess.run([exe], input=text, capture_output=True, text=True, timeout=60).stdout.split("\n")[:-1]
        assert len(out) == len(products)
        return [(KERNELS[int(a)], int(b), int(c)) for a, b, c in (r.split() for r in out)]

    return f


def layouts(products):
    return [(m, n, k, p) for m, n, k in products for p in ((0, 1) if k % 256 == 0 else (0,))]


def test_every_kernel_is_reached(ask):
    """Each kernel by a ragged product, with packed scales, with MX rows of whole stages and with a partial stage."""
    products = layouts(gpu.SMALL + gpu.LARGE + gpu.EVERY + gpu.PART + gpu.BIG)
    seen = set()
    for (m, n, k, packed), (kernel, _, _) in zip(products, ask(products)):
        tm, tn = TILE[kernel]
        seen.add((kernel, "packed" if packed else "stages" if k % 256 == 0 else "part", m % tm != 0 and n % tn != 0))
    for kernel in KERNELS:
        for layout in ("packed", "stages", "part"):
            assert (kernel, layout, True) in seen, (kernel, layout)


def test_big_tiles_every_way(ask):
    """The 256 x 256 kernel in both layouts: whole tiles and halves, each with rows of whole 16 bytes (bf16) and not."""
    products = layouts(gpu.BIG)
    seen = set()
    for (m, n, k, packed), (kernel, whole, halves) in zip(products, ask(products)):
        assert kernel == "256 x 256", (m, n, k, packed, kernel)
        for what, some in (("whole", whole), ("halves", halves)):
            if some:
                seen.add((packed, what, n % 8 == 0))
    assert seen == {(p, w, a) for p in (0, 1) for w in ("whole", "halves") for a in (True, False)}
    assert any(k % 256 == 128 for _, _, k in gpu.BIG)


def test_big_residuals(ask):
    in_place = layouts(gpu.BIG_IN_PLACE)
    streamed = layouts([s[:3] for s in gpu.BIG_STREAMED])
    assert all(r[0] == "256 x 256" for r in ask(in_place + streamed))
    for m, n, _, dt in gpu.BIG_STREAMED:
        assert m * n * (2 if dt == "bfloat16" else 4) >= 256 << 20


def test_choice_follows_the_measured_products(ask):
    """On the measured products (profiles/linear_products_by_kernel.md) the chosen kernel is hardly ever far from the
    fastest one."""
    products, times = [], []
    for row in open(os.path.join(ROOT, "profiles", "linear_products_by_kernel.md")):
        c = [x.strip() for x in row.strip().strip("|").split("|")]
        if c[0] in ("packed", "MX"):
            products.append((int(c[1]), int(c[2]), int(c[3]), int(c[0] == "packed")))
            times.append({k: float(t) for k, t in zip(KERNELS, c[4:]) if t})
    assert len(products) == 535
    loss = [t[kernel] / min(t.values()) for t, (kernel, _, _) in zip(times, ask(products))]
    assert sum(loss) / len(loss) < 1.015 and max(loss) < 1.36 and sum(x > 1.1 for x in loss) <= 23
