"""FastDiv / fdiv (csrc/kernels.h, csrc/device.h) against integer division over
everything that a call may ask of them: numerators up to 2^31 - 1 (the entries
of an expert order), divisors of 1 to 64 and any others.  No GPU needed."""
import os
import subprocess

import pytest

from test_fastdiv import CSRC, HIPCC, ROOT


@pytest.mark.skipif(not os.path.exists(HIPCC), reason="hipcc not found")
def test_division_is_exact_below_two_to_the_31(tmp_path):
    exe = str(tmp_path / "division_check")
    cmd = [HIPCC, "-O2", "-std=c++17", "-I" + CSRC, "-I" + os.path.join(ROOT, "include"),
           "--offload-arch=gfx950", "-x", "hip", os.path.join(ROOT, "tests", "division_check.cpp"), "-o", exe]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-2000:]
    out = subprocess.run([exe], capture_output=True, text=True, timeout=120)
    assert out.returncode == 0, out.stdout + out.stderr
    assert out.stdout.startswith("ok"), out.stdout
