"""GPU tests of lists of 4-bit copies on a stream of the caller's: copies,
results and tensors that are dropped right after the call, while it waits behind
that stream's work, and memory that is asked for at once."""

import pytest

torch = pytest.importorskip("torch")

import matrix_aware_optimizer_muon_amd as mm
from tests.test_gpu_mx4 import matrix

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]


def test_copies_dropped_behind_a_streams_work():
    xs = [matrix(2000, 1000, "f32"), matrix(700, 4100, "f32"), matrix(33, 65, "f32")]
    fixed = mm.Mx4Copies(xs)
    fixed.quantize()
    want = {axis: fixed.dequantize(axis=axis) for axis in (1, 0)}
    busy = torch.zeros(1 << 24, device="cuda")
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for axis in (1, 0, 1, 0):
        tensors = [x.clone() for x in xs]
        copies = mm.Mx4Copies(tensors)
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            for _ in range(100):
                busy.add_(1.0)
        copies.quantize(stream=side)
        got = copies.dequantize(axis=axis, stream=side)
        sizes = [copies._buffer.numel()] + [4 * t.numel() for t in tensors]
        del copies, tensors
        # the same sizes again on this stream, written before the side stream has come so far
        other = [torch.full((n,), 0x5A, dtype=torch.uint8, device="cuda") for n in sizes]
        torch.cuda.current_stream().wait_stream(side)
        assert torch.equal(got, want[axis])
        torch.cuda.synchronize()
        assert all(bool((t == 0x5A).all()) for t in other)
        del got, other
