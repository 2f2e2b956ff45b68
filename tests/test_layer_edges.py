"""The layer operators' host side at sizes of zero, on the CPU. Each query runs in a process of its
own, so that one that ends the process fails its test and not the run."""
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
QUERY = """
import ctypes, sys
import mxfp4_activation_quantizer_amd as kq
n = ctypes.c_int64(-1)
s = getattr(kq.lib(), sys.argv[1])(int(sys.argv[2]), int(sys.argv[3]), ctypes.byref(n))
print(s, n.value)
"""


@pytest.mark.parametrize("m,cols", [(5, 0), (0, 0), (0, 5), (2 ** 31 - 1, 0), (0, 2 ** 31 - 1)])
@pytest.mark.parametrize("name", ["kq_layernorm_backward_workspace_bytes", "kq_mxfp4_linear_backward_workspace_bytes"])
def test_no_workspace_for_no_elements(name, m, cols):
    p = subprocess.run([sys.executable, "-c", QUERY, name, str(m), str(cols)], capture_output=True, text=True, cwd=ROOT,
                       timeout=300)
    assert p.returncode == 0, "%s(%d, %d) ended the process: %d\n%s" % (name, m, cols, p.returncode, p.stderr)
    assert p.stdout.split() == ["0", "0"]
