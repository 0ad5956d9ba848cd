"""Which launches on 4-bit matrices go past the caches (CPU only;
`tests/host_mx4_stream/driver.cpp` on the library's own rule)."""

import os
import subprocess

import pytest

from matrix_aware_optimizer_muon_amd import build as B
from tests.test_debug_checks import HIPCC

HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.mark.skipif(not os.path.exists(HIPCC), reason="needs hipcc")
def test_by_the_bytes_of_the_values(tmp_path):
    exe = str(tmp_path / "driver")
    cmd = [HIPCC, "-O1", "-std=c++17", "-x", "hip", f"--offload-arch={B.ARCH}", f"-I{B.INCLUDE}", f"-I{B.CSRC}",
           os.path.join(HERE, "host_mx4_stream", "driver.cpp"), "-o", exe]
    r = subprocess.run(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)
    assert r.returncode == 0, r.stdout
    r = subprocess.run([exe], stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.stdout
