"""Properties of the compiled gfx950 code that the grouped kernels rely on
(CPU only: hipcc cross-compiles to assembly, nothing runs): their
direct-to-LDS loads set M0 in inline assembly, which is sound only while the
compiler keeps nothing of its own in M0."""
from __future__ import annotations

import os
import re
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HIPCC = shutil.which("hipcc") or "/opt/rocm/bin/hipcc"


def test_m0_only_set_for_lds_loads_of_the_grouped_kernels():
    if not os.path.exists(HIPCC):
        pytest.skip("hipcc not available")
    pkg = os.path.join(ROOT, "sample_gradient_clipping_layer_amd")
    out = subprocess.run([HIPCC, "--offload-arch=gfx950", "-O3", "-std=c++17", "-Xclang", "-target-feature", "-Xclang",
                          "-packed-fp32-ops", "-I", os.path.join(ROOT, "include"), "--cuda-device-only", "-S", "-o",
                          "-", os.path.join(pkg, "csrc", "dp_grouped.hip")], capture_output=True, text=True,
                         timeout=600)
    assert out.returncode == 0, out.stderr[-2000:]
    lines = [l.strip() for l in out.stdout.splitlines() if re.search(r"\bm0\b", l) and not l.strip().startswith(";")]
    assert len(lines) > 100, "expected the direct-to-LDS loads"
    other = [l for l in lines if not re.match(r"s_mov_b32 m0, (s\d+|vcc_lo|vcc_hi)$", l)]
    assert not other, other[:5]
