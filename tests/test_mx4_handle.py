"""The host code of microscaled 4-bit floats (CPU only): how lists are cut into
launches, a handle's 4-bit copies, activations, and every allocation failing in
turn (`tests/host_mx4/driver.cpp`, on the stand-ins of the handle's checks), as
built and under AddressSanitizer and UndefinedBehaviorSanitizer."""

import os
import shutil
import subprocess

import pytest

from matrix_aware_optimizer_muon_amd import build as BLD

HERE = os.path.dirname(os.path.abspath(__file__))
HIPCC = shutil.which("hipcc") or "/opt/rocm/bin/hipcc"
# sanitizers on the host side only (the device pass of a HIP compile takes none)
SAN = ["-Xarch_host", "-fsanitize=address", "-Xarch_host", "-fsanitize=undefined",
       "-Xarch_host", "-fno-sanitize-recover=all", "-Xarch_host", "-fno-omit-frame-pointer"]


def _run(cmd):
    r = subprocess.run(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)
    assert r.returncode == 0, r.stdout[-4000:]


@pytest.fixture(scope="module", params=["plain", "sanitized"])
def driver(request, tmp_path_factory):
    if not os.path.exists(HIPCC):
        pytest.skip("needs hipcc")
    d = tmp_path_factory.mktemp("mx4")
    san = SAN if request.param == "sanitized" else []
    objs = []
    for src in (os.path.join(BLD.CSRC, "muon_host.cpp"), os.path.join(HERE, "host_mx4", "driver.cpp")):
        objs.append(str(d / (os.path.splitext(os.path.basename(src))[0] + ".o")))
        _run([HIPCC, f"--offload-arch={BLD.ARCH}", "-O1", "-g", "-fPIC", "-std=c++17", "-x", "hip",
              "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops", *san,
              f"-I{BLD.INCLUDE}", f"-I{BLD.CSRC}", "-c", src, "-o", objs[-1]])
    exe = str(d / "mx4")
    link = ["-fsanitize=address", "-fsanitize=undefined"] if san else []
    _run([HIPCC, f"--offload-arch={BLD.ARCH}", "-fno-gpu-sanitize", *link, *objs, *BLD.LINK_FLAGS, "-o", exe])
    return exe


@pytest.mark.parametrize("what", ["launches", "weights", "acts", "exceptions"])
def test_mx4_host(driver, what):
    # the driver counts the ordinary operator new and leaves the nothrow one to the sanitizer
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=0:halt_on_error=1:alloc_dealloc_mismatch=0",
               UBSAN_OPTIONS="print_stacktrace=1:halt_on_error=1")
    r = subprocess.run([driver, what], stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True, timeout=300, env=env)
    assert r.returncode == 0 and r.stdout.splitlines()[-1:] == ["ok"], r.stdout[-4000:]
