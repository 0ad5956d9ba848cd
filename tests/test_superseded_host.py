"""Calls on a superseded static handle (CPU only; `tests/host_superseded/`)."""

import os
import subprocess

import pytest

from matrix_aware_optimizer_muon_amd import build as BLD
from tests.test_debug_checks import HIPCC

HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.mark.skipif(not os.path.exists(HIPCC), reason="needs hipcc")
def test_every_call_is_refused(tmp_path):
    exe = str(tmp_path / "driver")
    cmd = [HIPCC, f"--offload-arch={BLD.ARCH}", "-O1", "-g", "-std=c++17", "-x", "hip", f"-I{BLD.INCLUDE}", f"-I{BLD.CSRC}",
           os.path.join(BLD.CSRC, "muon_host.cpp"), os.path.join(HERE, "host_superseded", "driver.cpp"),
           *BLD.LINK_FLAGS, "-o", exe]
    r = subprocess.run(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)
    assert r.returncode == 0, r.stdout[-4000:]
    r = subprocess.run([exe], stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True, timeout=120)
    assert r.returncode == 0 and r.stdout.splitlines()[-1:] == ["ok"], r.stdout[-4000:]
