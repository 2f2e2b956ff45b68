"""The choice of kq_mxfp4_gated_linear's kernel just past a whole round of tiles and in a single round of large ones, on the CPU:
on the measured products (profiles/gated_products_by_kernel.md) the chosen kernel's time is near the fastest one's."""
import os

from tests import test_gated_choice as choice
from tests.test_gated_choice import ask  # noqa: F401  (fixture)


def measured():
    """[((m, n, k, packed), {kernel: us})]"""
    rows = []
    for row in open(os.path.join(choice.ROOT, "profiles", "gated_products_by_kernel.md")):
        c = [x.strip() for x in row.strip().strip("|").split("|")]
        if c[0] in ("packed", "MX"):
            rows.append(((int(c[1]), int(c[2]), int(c[3]), int(c[0] == "packed")),
                         {k: float(t) for k, t in zip(choice.KERNELS, c[4:]) if t != "-"}))
    return rows


def test_past_a_round(ask):  # noqa: F811
    """258, 264 and 516 tiles of 128 x 64 on 256 compute units, a round of 176 large tiles, whole and cut by n."""
    rows = [r for r in measured() if r[0][:2] in ((768, 2752), (1536, 1376), (1536, 2752), (768, 5504), (4096, 1376), (2048, 2752))]
    assert len(rows) >= 60
    for (product, times), (kernel, *_) in zip(rows, ask([r[0] for r in rows])):
        assert times[kernel] <= 1.1 * min(times.values()), (product, kernel, times)


def test_every_measured_product(ask):  # noqa: F811
    rows = measured()
    loss = [t[kernel] / min(t.values()) for (_, t), (kernel, *_) in zip(rows, ask([r[0] for r in rows]))]
    assert sum(loss) / len(loss) < 1.01 and max(loss) < 1.26 and sum(x > 1.1 for x in loss) <= 20
