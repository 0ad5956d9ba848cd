"""Host-only checks of how the binding sets the gradient norm and keeps its
buffer (no GPU): a recording stand-in for torch and for the library."""

import contextlib
import ctypes
import types

import pytest

torch = pytest.importorskip("torch")

from matrix_aware_optimizer_muon_amd import binding as B


class Recorder:
    """Stands in for torch and libmuon.so: the order of the calls."""

    def __init__(self, capturing=False):
        self.events = []
        stream = types.SimpleNamespace(synchronize=lambda: self.events.append("synchronize"), cuda_stream=0)
        self.cuda = types.SimpleNamespace(current_stream=lambda device=None: stream,
                                          is_current_stream_capturing=lambda: capturing,
                                          current_device=lambda: 0, device=lambda d: contextlib.nullcontext())

    def zeros(self, *shape, **kw):
        self.events.append("zeros")
        return torch.zeros(*shape)

    def muon_set_max_grad_norm(self, h, max_norm, norm_out):
        self.events.append(("set", max_norm.value if isinstance(max_norm, ctypes.c_float) else max_norm,
                            bool(norm_out.value if isinstance(norm_out, ctypes.c_void_p) else norm_out)))
        return B.MUON_OK

    def muon_destroy(self, h):
        return B.MUON_OK


def step_object(monkeypatch, norm_out=None, **kw):
    rec = Recorder(**kw)
    monkeypatch.setattr(B, "_torch", lambda: rec)
    st = object.__new__(B.MuonStep)
    st._lib, st._h, st.device = rec, ctypes.c_void_p(1), torch.device("cuda", 0)
    st._norm_out, st.grad_norm = norm_out, None
    return st, rec.events


def test_zero_fill_is_done_before_any_stream_can_step(monkeypatch):
    st, events = step_object(monkeypatch)
    st.set_max_grad_norm(0.5)
    assert events == ["zeros", "synchronize", ("set", 0.5, True)]
    # once: from then on the buffer is there
    st.set_max_grad_norm(0.0)
    st.set_max_grad_norm(float("inf"))
    assert events[3:] == [("set", 0.0, False), ("set", float("inf"), True)]
    st._h = None


def test_first_setting_is_refused_under_capture(monkeypatch):
    st, events = step_object(monkeypatch, capturing=True)
    with pytest.raises(RuntimeError, match="captur"):
        st.set_max_grad_norm(0.5)
    assert events == [] and st._norm_out is None and st.grad_norm is None
    st._h = None
    # with a buffer in place a captured program may set it
    st, events = step_object(monkeypatch, norm_out=torch.zeros(2), capturing=True)
    st.set_max_grad_norm(0.5)
    assert events == [("set", 0.5, True)]
    st._h = None


@pytest.mark.parametrize("max_norm", [1e-50, -1e-50, 1e39, 3.5e38, 10 ** 60])
def test_norms_that_float32_does_not_hold_are_refused(monkeypatch, max_norm):
    # the library would read 1e-50 as "off" and 1e39 as "measure only"
    st, events = step_object(monkeypatch, norm_out=torch.zeros(2))
    with pytest.raises(ValueError):
        st.set_max_grad_norm(max_norm)
    assert events == [] and st.grad_norm is None
    st._h = None


@pytest.mark.parametrize("max_norm,on", [(0, False), (0.0, False), (1e-45, True), (2.0 ** -126, True), (3, True),
                                         (3.4e38, True), (float("inf"), True), (torch.tensor(0.25), True)])
def test_norms_that_float32_holds_are_set(monkeypatch, max_norm, on):
    st, events = step_object(monkeypatch, norm_out=torch.zeros(2))
    st.set_max_grad_norm(max_norm)
    assert events == [("set", ctypes.c_float(float(max_norm)).value, on)]
    assert (st.grad_norm is not None) == on == (events[0][1] > 0)
    st._h = None
