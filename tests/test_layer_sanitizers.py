"""The host side of the layer norm's and kq_mxfp4_linear's entry points under AddressSanitizer and
UndefinedBehaviorSanitizer on the CPU (no GPU): argument checks at the extremes of int64 sizes."""
import os
import subprocess

import pytest

SAN = os.path.join(os.path.dirname(os.path.abspath(__file__)), "sanitize")
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
CLANG = "/opt/rocm/llvm/bin/clang"
# sanitizers on the host pass only
HOST_SAN = "-Xarch_host -fsanitize=address -Xarch_host -fsanitize=undefined -Xarch_host -fno-sanitize-recover=all".split()
ENV = dict(os.environ, ASAN_OPTIONS="detect_leaks=0:abort_on_error=1", UBSAN_OPTIONS="halt_on_error=1")


def run(cmd, **kw):
    p = subprocess.run(cmd, capture_output=True, text=True, **kw)
    assert p.returncode == 0, "%s\n%s\n%s" % (" ".join(cmd), p.stdout[-4000:], p.stderr[-4000:])
    return p


@pytest.mark.skipif(not os.path.exists(HIPCC) or not os.path.exists(CLANG), reason="ROCm toolchain not found")
def test_layer_host_checks_under_asan_ubsan(tmp_path):
    from mxfp4_activation_quantizer_amd import build as kqbuild
    lib = str(tmp_path / "liblayer_san.so")
    flags = [f for f in kqbuild.HIP_FLAGS if f != "-O3"] + ["-O1", "-g"]
    parts = [os.path.join(kqbuild.CSRC, f) for f in ("kq_norm.hip", "kq_linear.hip", "kq_gemm256.hip")]
    run([HIPCC, *flags, *HOST_SAN, "-I", kqbuild.INCLUDE, "-I", kqbuild.CSRC, *parts, "-o", lib])
    exe = str(tmp_path / "layer_checks")
    run([CLANG, "-O1", "-g", "-fsanitize=address,undefined", "-fno-sanitize-recover=all", "-fno-omit-frame-pointer",
         "-I", kqbuild.INCLUDE, os.path.join(SAN, "layer_checks_driver.c"), "-L", str(tmp_path), "-llayer_san",
         "-Wl,-rpath," + str(tmp_path), "-lm", "-o", exe])
    assert "ok" in run([exe], env=ENV).stdout
