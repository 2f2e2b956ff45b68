"""A host helper called before torch is imported: the process still has one HIP runtime (of two, the library's own would
see no device, and every later launch would be refused)."""
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SCRIPT = """
import mxfp4_activation_quantizer_amd as kq
assert kq.rope_frequencies(8).shape == (4,)
import torch
print(sorted({os.path.realpath(line.split()[-1]) for line in open("/proc/self/maps") if "libamdhip64" in line}))
print("launch", torch.cuda.is_available() and int(kq.quantize_mxfp4(torch.ones(1, 32, dtype=torch.bfloat16, device="cuda"))[1][0, 0]))
"""


def run():
    p = subprocess.run([sys.executable, "-c", "import os\n" + SCRIPT], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert p.returncode == 0, p.stderr[-2000:]
    return p.stdout.split("\n")


def test_one_hip_runtime():
    assert run()[0].count("libamdhip64") == 1


@pytest.mark.gpu
def test_launch_after_a_host_helper():
    # a block of ones: its largest is 1 = 2^0, so the scale is 2^(0 - 2)
    assert run()[1] == "launch 125"
