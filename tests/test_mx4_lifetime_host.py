"""Host-only checks (no GPU) of how long a handle holds the 4-bit copies that its
steps renew: until they are replaced, with the allocator told of the steps'
streams, or as long as the handle once a step has been captured with them."""

import contextlib
import ctypes
import gc
import types
import weakref

import pytest

torch = pytest.importorskip("torch")

from matrix_aware_optimizer_muon_amd import binding as B


class Copies:
    """Stands in for Mx4Copies."""

    _descs, _n = None, 1

    def __init__(self):
        self.told = []

    def record_stream(self, stream):
        self.told.append(stream)


class World:
    """Torch and the library: the current stream, whether it is being captured, and what the library answers."""

    def __init__(self):
        self.stream, self.capturing, self.status, self.steps = 0, set(), B.MUON_OK, []
        self.cuda = types.SimpleNamespace(
            current_device=lambda: 0, device=lambda d: contextlib.nullcontext(), stream=self.on,
            current_stream=lambda device=None: types.SimpleNamespace(cuda_stream=self.stream),
            is_current_stream_capturing=lambda: self.stream in self.capturing,
            ExternalStream=lambda raw, device=None: raw, default_stream=lambda device=None: "default")

    @contextlib.contextmanager
    def on(self, stream):
        before, self.stream = self.stream, stream.cuda_stream
        yield
        self.stream = before

    def muon_set_mx4_weights(self, h, descs, n):
        return self.status

    def muon_step(self, h, lr, stream):
        self.steps.append(stream.value or 0)
        return B.MUON_OK

    def muon_last_error(self):
        return b"refused"

    muon_status_str = muon_last_error

    def muon_destroy(self, h):
        return B.MUON_OK


@pytest.fixture
def world(monkeypatch):
    w = World()
    monkeypatch.setattr(B, "_torch", lambda: w)
    return w


def handle(world):
    st = object.__new__(B.MuonStep)
    st._lib, st._h, st._keep, st._raw_stream = world, ctypes.c_void_p(1), [], None
    st.device = torch.device("cuda", 0)
    return st


def side(raw):
    return types.SimpleNamespace(cuda_stream=raw)


def test_replaced_copies_go(world):
    st = handle(world)
    refs = []
    for k in range(5):
        c = Copies()
        refs.append(weakref.ref(c))
        st.set_mx4_weights(c)
        st.step(), st.step(stream=side(77)), st.step()
        told = c.told
        del c
        gc.collect()
        assert [r() is not None for r in refs] == [False] * k + [True]
        st.set_mx4_weights(Copies() if k % 2 else None)
        gc.collect()
        assert refs[-1]() is None and sorted(told, key=str) == [77, "default"]
    assert st._keep == [] and world.steps == [0, 77, 0] * 5
    st._h = None


@pytest.mark.parametrize("given", [False, True])
def test_captured_copies_stay(world, given):
    """Captured on the current stream, or on one that the step is given."""
    st = handle(world)
    world.capturing = {5}
    a, b = Copies(), Copies()
    ra, rb = weakref.ref(a), weakref.ref(b)
    st.set_mx4_weights(a)
    st.step()
    if given:
        st.step(stream=side(5)), st.step(stream=side(5))
    else:
        with world.on(side(5)):
            st.step(), st.step()
    st.set_mx4_weights(b)
    st.step(stream=side(6))
    st.set_mx4_weights(a), st.set_mx4_weights(a)
    st.step()
    st.set_mx4_weights(None)
    del a, b
    gc.collect()
    assert ra() is not None and rb() is None and len(st._keep) == 1
    st._h = None


def test_a_refused_list_leaves_the_one_that_was_set(world):
    st = handle(world)
    a, b = Copies(), Copies()
    st.set_mx4_weights(a)
    world.status = 1
    with pytest.raises(B.MuonError):
        st.set_mx4_weights(b)
    assert st._mx4 is a and a.told == []
    st._h = None
