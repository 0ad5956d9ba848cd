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


def test_replaced_copies_behind_a_streams_steps():
    """Copies that are replaced and dropped while a step that renews them waits behind its stream's work: memory that
    is asked for at once is not theirs yet, and all of it comes back."""
    gen = torch.Generator(device="cuda").manual_seed(2)
    w, g = (torch.randn(1500, 2000, generator=gen, device="cuda") for _ in range(2))
    m, v = torch.zeros_like(w), torch.zeros_like(w)
    opt = mm.MuonStep([mm.adam_tensor_desc(w, g, m, v)], mm.default_hparams(), keepalive=[g, m, v])
    busy = torch.zeros(1 << 24, device="cuda")
    side = torch.cuda.Stream()
    kept = mm.Mx4Copies([w])
    torch.cuda.synchronize()
    memory = []
    for given in (True, False) * 4:
        copies = mm.Mx4Copies([w])
        size = copies._buffer.numel()
        opt.set_mx4_weights(copies)
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            for _ in range(100):
                busy.add_(1.0)
            if not given:
                opt.step()
        if given:
            opt.step(stream=side)
        opt.set_mx4_weights(kept)
        del copies
        other = torch.full((size,), 0x5A, dtype=torch.uint8, device="cuda")
        torch.cuda.synchronize()
        assert bool((other == 0x5A).all())
        del other
        memory.append(torch.cuda.memory_allocated())
    assert memory[-1] == memory[1]
    # captured ones stay: the graph writes to them
    captured = mm.Mx4Copies([w])
    opt.set_mx4_weights(captured)
    opt.step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        opt.step()
    at = captured._buffer.data_ptr()
    opt.set_mx4_weights(None)
    del captured
    others = [torch.full((size,), 0x5A, dtype=torch.uint8, device="cuda") for _ in range(8)]
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert all(t.data_ptr() != at and bool((t == 0x5A).all()) for t in others)
    assert opt.flags() == 0
    opt.close()
