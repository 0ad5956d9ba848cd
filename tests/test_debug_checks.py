"""What the debug build (MUON_DEBUG_BOUNDS=1) adds: every kernel that takes its
work from a task list of the plan checks the task, and raises flag bit 2 where
it would leave its tensor.  Compiles the sources both ways and counts the
kernels that hold more flag atomics (CPU only)."""

import os
import re
import shutil
import subprocess

import pytest

from matrix_aware_optimizer_muon_amd import build as B

HIPCC = shutil.which("hipcc") or "/opt/rocm/bin/hipcc"


def _atomics(src, out, *flags):
    subprocess.run([HIPCC, *B.HIP_FLAGS, *flags, "--cuda-device-only", "-S", f"-I{B.INCLUDE}",
                    os.path.join(B.CSRC, src), "-o", out], check=True, stdout=subprocess.PIPE, stderr=subprocess.STDOUT)
    with open(out) as f:
        kernels = re.split(r"\n(?=_Z\S+:)", f.read())[1:]
    return {k.split(":", 1)[0]: len(re.findall(r"\b(?:global|flat)_atomic_or\b", k)) for k in kernels}


@pytest.mark.skipif(not os.path.exists(HIPCC), reason="needs hipcc")
@pytest.mark.parametrize("src,kernels", [("elementwise.hip", ("momentum_kernel", "update_kernel")),
                                         ("adamw_packed.hip", ("adamw_packed_kernel", "unpack_kernel", "pack_kernel")),
                                         ("grad_norm.hip", ("grad_norm_kernel",))])
def test_debug_build_checks_every_task(tmp_path, src, kernels):
    release = _atomics(src, str(tmp_path / "release.s"))
    debug = _atomics(src, str(tmp_path / "debug.s"), *B.DEBUG_FLAGS)
    assert release.keys() == debug.keys()
    for kernel in kernels:
        names = [n for n in debug if kernel in n]
        assert names, kernel
        without = [n for n in names if debug[n] <= release[n]]
        assert not without, f"no check in {without}"
