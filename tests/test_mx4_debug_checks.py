"""The debug build checks which part of the second moment a block takes, and its
room for partial sums; nothing else of the 4-bit kernels takes its work from the
host's tables (CPU only)."""

import os

import pytest

from matrix_aware_optimizer_muon_amd import build as B
from tests.test_debug_checks import HIPCC, _atomics


@pytest.mark.skipif(not os.path.exists(HIPCC), reason="needs hipcc")
def test_debug_build_checks_every_tile(tmp_path):
    release = _atomics("mx4_moment.hip", str(tmp_path / "release.s"))
    debug = _atomics("mx4_moment.hip", str(tmp_path / "debug.s"), *B.DEBUG_FLAGS)
    assert release.keys() == debug.keys()
    tiles = [n for n in debug if "tile_kernel" in n]
    assert len(tiles) == 3 and all(debug[n] > release[n] for n in tiles)
