"""Host-only check that every call of a handle reaches the library with the
handle's device the current one (no GPU): HIP launches, and the default
stream, are the current device's."""

import contextlib
import ctypes
import types

import pytest

torch = pytest.importorskip("torch")

from matrix_aware_optimizer_muon_amd import binding as B
from tests.test_binding_host import _FakeActs, _FakeStream


class World:
    """Two devices, and a library that notes the current one of each call."""

    def __init__(self):
        self.current, self.calls = 0, []
        self.cuda = types.SimpleNamespace(current_device=lambda: self.current, device=self.device,
                                          current_stream=lambda device=None: _FakeStream(),
                                          is_current_stream_capturing=lambda: False)
        self.float32, self.bfloat16 = torch.float32, torch.bfloat16

    @contextlib.contextmanager
    def device(self, device):
        before, self.current = self.current, device.index
        yield
        self.current = before

    def __getattr__(self, name):
        def call(*args):
            self.calls.append((name, self.current))
            return b"adamw" if name == "muon_phase_name" else B.MUON_OK
        return call


CALLS = {
    "step": lambda st: st.step(),
    "step_timed": lambda st: st.step_timed(),
    "refresh": lambda st: st.precond_refresh(0, 0, _FakeActs([])),
    "accumulate": lambda st: st.precond_accumulate(0, 0, _FakeActs([])),
    "refresh_accumulated": lambda st: st.precond_refresh_accumulated(0, 0),
    "set_adam_step": lambda st: st.set_adam_step(3),
    "adam_step": lambda st: st.adam_step(),
    "flags": lambda st: st.flags(reset=True),
    "close": lambda st: st.close(),
}


@pytest.mark.parametrize("index", [0, 1])
@pytest.mark.parametrize("name", CALLS)
def test_calls_run_on_the_handles_device(monkeypatch, name, index):
    world = World()
    monkeypatch.setattr(B, "_torch", lambda: world)
    st = object.__new__(B.MuonStep)
    st._lib, st._h, st._keep = world, ctypes.c_void_p(1), []
    st.device, st._raw_stream = torch.device("cuda", index), None
    CALLS[name](st)
    made = [c for c in world.calls if c[0] != "muon_phase_name"]
    assert len(made) == 1 and made[0][1] == index and world.current == 0
    st._h = None
