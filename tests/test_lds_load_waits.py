"""gfx9 needs one wait state between a scalar instruction that writes M0 and a
load to LDS, which takes its place from M0.  hipcc puts it behind its own
writes, not into inline assembly, so every load to LDS in the kernels' code is
looked at here (CPU only)."""

import os
import re
import subprocess

import pytest

from matrix_aware_optimizer_muon_amd import build as B
from tests.test_debug_checks import HIPCC

WRITES_M0 = re.compile(r"s_\w+\s+m0,")
LOADS_TO_LDS = re.compile(r"(global|buffer|scratch)_load_lds_|buffer_load_\w+ .*\blds\b")


def unprotected(asm):
    """The loads to LDS that directly follow a write of M0."""
    code = [line.split(";")[0].strip() for line in asm.splitlines()]
    code = [line for line in code if line and not line.startswith(".") and not line.endswith(":")]
    loads = [k for k, line in enumerate(code) if LOADS_TO_LDS.match(line)]
    return len(loads), [code[k - 1] + " / " + code[k] for k in loads if WRITES_M0.match(code[k - 1])]


def test_what_is_looked_for():
    bad = "\ts_mov_b32 m0, s4\n\tglobal_load_lds_dwordx4 v1, s[4:5]\n"
    assert unprotected(bad) == (1, ["s_mov_b32 m0, s4 / global_load_lds_dwordx4 v1, s[4:5]"])
    assert unprotected(bad.replace("\n\tglobal", "\n\t;;#ASMEND\n.LBB0_1:\n\tglobal"))[1]
    assert unprotected(bad.replace("\n\tglobal", "\n\ts_nop 0\n\tglobal")) == (1, [])


@pytest.mark.skipif(not os.path.exists(HIPCC), reason="needs hipcc")
@pytest.mark.parametrize("src", [s for s in B.SOURCES if s.endswith(".hip")])
def test_a_wait_state_between_m0_and_the_load(tmp_path, src):
    out = str(tmp_path / "k.s")
    subprocess.run([HIPCC, *B.HIP_FLAGS, "--cuda-device-only", "-S", f"-I{B.INCLUDE}", os.path.join(B.CSRC, src),
                    "-o", out], check=True, stdout=subprocess.PIPE, stderr=subprocess.STDOUT)
    with open(out) as f:
        loads, bad = unprotected(f.read())
    assert (loads > 0) == (src in ("ns_gemm.hip", "mx4_moment.hip"))
    assert not bad, f"{len(bad)} of {loads}: {bad[:3]}"
