"""Host-only check (no GPU) that calls on a stream of the caller's tell torch's
allocator of every tensor whose memory that stream uses: what is dropped right
after the call must not be handed out again before the stream is done."""

import contextlib
import types

import pytest

torch = pytest.importorskip("torch")

from matrix_aware_optimizer_muon_amd import binding as B


@pytest.fixture
def world(monkeypatch):
    """Tensors on the CPU, a library that does nothing, and what streams were told to the allocator."""
    seen = []
    monkeypatch.setattr(torch.Tensor, "record_stream",
                        lambda t, s: seen.append((t.untyped_storage().data_ptr(), s)), raising=False)
    monkeypatch.setattr(torch.cuda, "stream", lambda s: contextlib.nullcontext())
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: "current")
    monkeypatch.setattr(B, "_raw_stream", lambda device, stream: 0)
    monkeypatch.setattr(B, "_launch_on", lambda device, function, *args: None)
    monkeypatch.setattr(B, "load_library", lambda: types.SimpleNamespace(muon_mx4_quantize=None, muon_mx4_dequantize=None))
    return seen


def memory(*tensors):
    return [t.untyped_storage().data_ptr() for t in tensors]


def test_copies_and_their_tensors(world):
    tensors = [torch.zeros(40, 70), torch.zeros(3, 5, dtype=torch.bfloat16)]
    copies = B.Mx4Copies(tensors)
    (held,) = {t.untyped_storage().data_ptr() for c in copies.copies for f in c for t in (f.codes, f.scales)}
    copies.quantize(stream="side")
    assert {("side", at) for at in [held] + memory(*tensors)} == {(s, at) for at, s in world}
    world.clear()
    out = copies.dequantize(axis=0, stream="side")       # of that stream's memory, and used on the current one
    assert sorted(world, key=str) == sorted([(held, "side"), (memory(out)[0], "current")], key=str)
    world.clear()
    copies.dequantize(out=out, stream="side")
    assert set(world) == {(held, "side"), (memory(out)[0], "side")}
    world.clear()
    copies.quantize(), copies.dequantize()
    assert world == []


def test_single_matrices(world):
    x = torch.zeros(40, 70)
    q = B.mx4_quantize(x, stream="side")
    assert set(world) == {(memory(x)[0], "side")} | {(at, "current") for at in memory(q.codes, q.scales)}
    world.clear()
    out = B.mx4_dequantize(q, stream="side")
    assert set(world) == {(at, "side") for at in memory(q.codes, q.scales)} | {(memory(out)[0], "current")}
