"""The accuracy that csrc/kq_turn.hpp states for the rotation's sine and cosine, on the CPU: a host-only build of the
function, in the library's own floating-point mode, scanned by tests/native/turn_check.cpp."""
import os
import subprocess

import pytest

from mxfp4_activation_quantizer_amd import build as kqbuild

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.skipif(not os.path.exists(kqbuild.HIPCC), reason="hipcc not found")
def test_sine_and_cosine(tmp_path):
    exe = str(tmp_path / "turn_check")
    p = subprocess.run([kqbuild.HIPCC, "-x", "hip", "--cuda-host-only", "-std=c++17", "-O2", "-mfma", "-ffp-contract=off",
                        "-I", kqbuild.CSRC, os.path.join(ROOT, "tests", "native", "turn_check.cpp"), "-o", exe],
                       capture_output=True, text=True)
    assert p.returncode == 0, p.stderr[-2000:]
    p = subprocess.run([exe], capture_output=True, text=True, timeout=300)
    assert p.returncode == 0
    sine, cosine = (float(x) for x in p.stdout.split())
    # half a unit for the angle's rounding (times x cot x <= 1), half for the last sum, the rest the series' own
    assert 0.5 < sine <= 1.5 and 0.5 < cosine <= 1.25
