"""bench.py's line on stdout: whole where only the last 8000 characters of the output are kept."""
import json

import bench


def stats(i):
    return {"m": 18432, "d": 12288, "median_us": 100.123 + i, "mean_us": 101.456, "p10_us": 99.123, "p90_us": 103.789,
            "GBps": 5678.9, "Gelem_per_s": 2345.67, "pct_hbm_peak": 67.8}


def result(shapes):
    kinds = ("quantize", "smoothquant", "fused", "fwht")
    return {"metric": "m", "value": 1.0, "unit": "GB/s", "n_gpus": 1, "config": {"workload": "w"},
            "kernels": {k: [stats(0), stats(1)] for k in kinds[:3]},
            "extras": {"table": {"shape_%dx12288" % i: dict({k: stats(i) for k in kinds}, ratio=0.5) for i in range(shapes)},
                       "form": [stats(3), stats(4)], "fold": dict(stats(5), note="a note"), "layer": {"a_us": 1.5}}}


def test_the_line_has_the_medians_and_fits():
    out = result(30)
    assert len(json.dumps(out)) > 8000  # as it was printed before, cut at its beginning
    line = bench.headline(out)
    assert len(line) <= bench.LINE_LIMIT < 8000 and "\n" not in line
    got = json.loads(line)
    assert {k: v for k, v in got.items() if k != "extras"} == {k: v for k, v in out.items() if k != "extras"}
    assert got["extras"]["table"]["shape_7x12288"] == {"quantize": 107.123, "smoothquant": 107.123, "fused": 107.123,
                                                       "fwht": 107.123, "ratio": 0.5}
    assert got["extras"]["form"] == [103.123, 104.123] and got["extras"]["fold"] == 105.123
    assert got["extras"]["layer"] == {"a_us": 1.5}


def test_a_line_that_would_not_fit_leaves_the_extras_out():
    out = result(300)
    line = bench.headline(out)
    assert len(line) <= bench.LINE_LIMIT
    assert json.loads(line) == {k: v for k, v in out.items() if k != "extras"}


def test_without_extras_nothing_changes():
    out = {k: v for k, v in result(1).items() if k != "extras"}
    assert json.loads(bench.headline(out)) == out
